// The dense layer's product for few rows (tokens of a batch that decodes): B's way through
// the memory bounds it.  A warp takes B from global memory straight into the registers of
// mma.sync, sixteen bytes a lane: the sum's order is free, so lane t of four takes eight
// neighbours of it from B and A alike, and no operand passes shared or tensor memory.
//   B stored [N][K]   a warp 32 rows of B, 64 places of the sum a step
//   B stored [K][N]   a warp 64 columns of B, 32 places a step, paired by byte permutes
// The sum is cut among a block's eight warps and among a cluster's blocks, which add what
// they have through shared memory, in their order.
// One row of 2048 by [8192][2048] bf16 takes 7.6 us (33.5 MB at 4.4 TB/s, the launch and the
// ramp of one wave among it), eight 7.7, sixteen 10.2 (A's words take as many registers as
// B's); [K][N] 9.4, 9.7 and 12.5, where sixteen rows read B twice.  Those are weights from HBM,
// 600 MB of them in turn; where L2 holds B, 4.2, 4.6 and 8.3 us.  8 x 4096 x 1024 takes 4.0 us
// (2.8 from L2), 8 x 768 x 768 3.2 (2.3).  A in shared memory, staged for two steps of all
// warps at a time, took 10.3 and 14.6 us for eight and sixteen rows.
#include <type_traits>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

struct FewArgs {
  Mat a, b;
  int M, N, K;
  int cut, per;        // blocks of a cluster, and the places of the sum of each
  Epilogue ep;
};

template <typename T>
__device__ __forceinline__ void finish(const Epilogue& e, float z, int64_t m, int64_t n) {
  if (e.bias) z += to_f32(static_cast<const T*>(e.bias)[n]);
  if (e.z.data) static_cast<T*>(e.z.data)[m * e.z.ld + n] = from_f32<T>(z);
  float y = 0.0f;
  by_act(e.act, [&](auto act) { y = act_of<decltype(act)::value>(z); });
  if (e.residual.data) y += to_f32(static_cast<const T*>(e.residual.data)[m * e.residual.ld + n]);
  static_cast<T*>(e.out.data)[m * e.out.ld + n] = from_f32<T>(y);
}

// The 16 bytes of a row of `n` elements from `at` on, which hold one of them at least, or 0.
template <typename T>
__device__ __forceinline__ uint4 word_of(const T* row, int at, int n) {
  return at < n ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0, 0, 0, 0);
}

// u without what is past its first `keep` elements.
__device__ __forceinline__ uint4 head_of(const uint4& u, int keep) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = keep >= 2 * i + 2 ? w[i] : keep == 2 * i + 1 ? w[i] & 0xffffu : 0u;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// D[16][8] += A[16][16] B[16][8].
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float cluster_ld(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(addr, rank)));
  return v;
}

// A block's columns of the output, and the places of the sum of a warp's step.
template <bool KN>
constexpr int kCols = KN ? 64 : 32;
template <bool KN>
constexpr int kStep = KN ? 32 : 64;
template <bool KN>
constexpr int kPitch = kCols<KN> + 4;

template <bool KN, int TILES>
constexpr int kFewBytes = kWarps * 8 * TILES * kPitch<KN> * 4;

// TILES: of eight rows of A.
template <typename T, bool KN, int TILES>
__global__ void __launch_bounds__(kThreads, 2) k_few(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(16) float red[];  // [warp][row of A][column]
  constexpr int COLS = kCols<KN>, STEP = kStep<KN>, PITCH = kPitch<KN>, ROWS = 8 * TILES;
  constexpr int kAcross = COLS / 16;  // tiles of sixteen columns
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % a.cut;
  const int n0 = blockIdx.x / a.cut * COLS, m0 = blockIdx.y * ROWS, rows = min(a.M - m0, ROWS);
  const T* x = static_cast<const T*>(a.a.data) + (m0 + g) * a.a.ld + 8 * t;
  const T* b = static_cast<const T*>(a.b.data) + (KN ? 8 * t * a.b.ld + n0 + 8 * g : (n0 + g) * a.b.ld + 8 * t);
  const int begin = rank * a.per, end = min(a.K, begin + a.per);
  float sum[kAcross][TILES][4];
#pragma unroll
  for (int i = 0; i < kAcross; ++i)
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[i][j][k] = 0.0f;
  // A lane's words of a step.  B's: [N][K] rows g, g + 8, g + 16, g + 24 of two halves of
  // 32 places; [K][N] the columns from 8 g of places 8 t to 8 t + 7.
  constexpr int kHalves = STEP / 32;
  struct Words {
    uint4 w[8], v[kHalves][TILES];
  };
  auto load = [&](Words& to, int k0) {
    uint4(&w)[8] = to.w;
    const T* p = b + (KN ? k0 * a.b.ld : k0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = make_uint4(0, 0, 0, 0);
      if (KN) {
        if (k0 + 8 * t + i < end) w[i] = word_of(p + i * a.b.ld, 0, a.N - n0 - 8 * g);
      } else {
        if (n0 + g + 8 * (i & 3) < a.N)
          w[i] = word_of(p + 8 * (i & 3) * a.b.ld, 32 * (i >> 2), end - k0 - 8 * t);
      }
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        to.v[h][j] = make_uint4(0, 0, 0, 0);
        if (8 * j + g < rows) to.v[h][j] = word_of(x + 8 * j * a.a.ld + k0, 32 * h, end - k0 - 8 * t);
      }
    if (k0 < end && k0 + STEP > end) {  // the sum may end inside a word
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!KN) w[i] = head_of(w[i], end - k0 - 8 * t - 32 * (i >> 2));
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int j = 0; j < TILES; ++j) to.v[h][j] = head_of(to.v[h][j], end - k0 - 8 * t - 32 * h);
    }
  };
  auto multiply = [&](const Words& from) {
    const uint4(&w)[8] = from.w;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const uint4(&v)[TILES] = from.v[h];
#pragma unroll
      for (int i = 0; i < kAcross; ++i) {
        uint4 p, q;  // of the tile's columns g and g + 8
        if (KN) {    // columns 8 g + 2 i and 8 g + 2 i + 1, places in pairs
          uint32_t u[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) u[k] = i == 0 ? w[k].x : i == 1 ? w[k].y : i == 2 ? w[k].z : w[k].w;
          p = make_uint4(__byte_perm(u[0], u[1], 0x5410), __byte_perm(u[2], u[3], 0x5410),
                         __byte_perm(u[4], u[5], 0x5410), __byte_perm(u[6], u[7], 0x5410));
          q = make_uint4(__byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632),
                         __byte_perm(u[4], u[5], 0x7632), __byte_perm(u[6], u[7], 0x7632));
        } else {
          p = w[4 * h + 2 * i];
          q = w[4 * h + 2 * i + 1];
        }
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          mma<T>(sum[i][j], p.x, q.x, p.y, q.y, v[j].x, v[j].y);
          mma<T>(sum[i][j], p.z, q.z, p.w, q.w, v[j].z, v[j].w);
        }
      }
    }
  };
  grid_wait();
  // two steps are under way at a time
  constexpr int kStride = kWarps * STEP;
  Words one, two;
  int k0 = begin + warp * STEP;
  load(one, k0);
#pragma unroll 1
  for (; k0 < end; k0 += 2 * kStride) {
    load(two, k0 + kStride);
    multiply(one);
    load(one, k0 + 2 * kStride);
    multiply(two);
  }
  float* mine = red + warp * ROWS * PITCH;
#pragma unroll
  for (int i = 0; i < kAcross; ++i)
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = KN ? 8 * g + 2 * i + (k >> 1) : 16 * i + g + 8 * (k >> 1);
        mine[(8 * j + 2 * t + (k & 1)) * PITCH + col] = sum[i][j][k];
      }
  __syncthreads();
  auto at = [&](int i) { return i / COLS * PITCH + i % COLS; };
  for (int i = threadIdx.x; i < rows * COLS; i += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) s += red[q * ROWS * PITCH + at(i)];
    if (a.cut > 1)
      red[at(i)] = s;
    else if (n0 + i % COLS < a.N)
      finish<T>(a.ep, s, m0 + i / COLS, n0 + i % COLS);
  }
  if (a.cut == 1) return;
  cluster_sync();
  const uint32_t base = smem_u32(red);
  for (int i = rank * kThreads + threadIdx.x; i < rows * COLS; i += kThreads * a.cut) {
    float s = 0.0f;
    for (int q = 0; q < a.cut; ++q) s += cluster_ld(base + 4 * at(i), q);
    if (n0 + i % COLS < a.N) finish<T>(a.ep, s, m0 + i / COLS, n0 + i % COLS);
  }
  cluster_sync();  // a block's shared memory stays until all have read it
}

template <typename T, bool KN, int TILES>
cudaError_t go(const Gemm& g, cudaStream_t s) {
  FewArgs a{};
  a.a = g.a;
  a.b = g.b;
  a.N = (int)g.N;
  a.K = (int)g.K;
  a.M = (int)g.M;
  a.ep = g.ep;
  const int64_t across = (g.N + kCols<KN> - 1) / kCols<KN>, down = (g.M + 8 * TILES - 1) / (8 * TILES);
  // Blocks of a cluster: as two blocks an SM leave room for, while every warp has two steps
  // (a cluster's start and its waits take some 1.3 us: 768 x 768 2.2 us whole, 3.4 cut).
  a.cut = 1;
  while (a.cut < 8 && across * down * a.cut <= 152 && a.K > 2 * kWarps * a.cut * kStep<KN>) a.cut *= 2;
  a.per = (a.K + a.cut * kStep<KN> - 1) / (a.cut * kStep<KN>) * kStep<KN>;
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_few<T, KN, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kFewBytes<KN, TILES>);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(across * a.cut), (unsigned)down);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = kFewBytes<KN, TILES>;
  c.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.cut;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = a.cut > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, k_few<T, KN, TILES>, a);
}

}  // namespace

// Up to 16 rows this is the quicker way for any B (weights from HBM, us here and on tiles of
// the matrix unit: 16 x 8192 x 2048 bf16 10.2 and 13.4, by [K][N] weights 12.5 and 14.2; 16 x
// 2048 x 8192 11.8 and 19.9, 13.8 and 19.6).  Up to 128 where what is read, B for every 16 rows
// (by [K][N] weights for every eight), is less than the tiles' start and end are worth: 64 x 2048
// x 1024 5.7 and 8.9, [K][N] 7.0 and 9.4; 48 x 4096 x 1024 would take 9.9 and 9.0, 10.6 and 9.5.
// Twice as much along a long sum, which the tiles cut and join: 64 x 1024 x 4096 10.9 and 17.5,
// 13.0 and 17.3; 128 x 1024 x 2048 8.6 and 12.6, 11.7 and 12.6.  One limit holds for both layouts.
// Where a backward pass can put both products in one launch, those with a short sum stay on
// the tiles from 17 rows on (128 x 768 x 768: 12.2 us together, 15.6 apart); dx alone does too,
// as the workspace's size is asked for without knowing which are wanted.
bool few_rows(int64_t M, int64_t N, int64_t K, bool a_mn, bool pair) {
  if (a_mn || M > 128 || (M > 16 && pair && K < 2048)) return false;
  return M <= 16 || (M + 15) / 16 * N * K <= (K < 2048 ? 1 << 23 : 1 << 24);
}

cudaError_t launch_few(const Gemm& g, cudaStream_t s) {
  auto by_rows = [&](auto zero, auto kn) {
    using T = decltype(zero);
    constexpr bool KN = decltype(kn)::value;
    if constexpr (!KN)
      if (g.M > 8) return go<T, KN, 2>(g, s);
    return go<T, KN, 1>(g, s);
  };
  auto by_layout = [&](auto zero) {
    return g.b_mn ? by_rows(zero, std::true_type()) : by_rows(zero, std::false_type());
  };
  return g.ep.type == OB_TYPE_BF16 ? by_layout(__nv_bfloat16()) : by_layout(__half());
}

}  // namespace ob
