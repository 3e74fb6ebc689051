// One product of the dense layer on the tensor cores, with its epilogue.
//
// Workers stay and take unit after unit of the output: a pair of blocks a tile
// of 256 x 256 (each holds 128 rows of A and of the sum, and half of B), or, where
// that leaves most of the card idle, a block a tile of 128 x 128.  In a block one
// warp issues the copies (tiles of 64 along the sum, 128-byte swizzle, either
// operand stored along the sum or across it), one the products, and sixteen
// take the sums out of tensor memory, a row a lane: bias, activation, residual, one
// rounding.  They store through shared memory and TMA, 32 x 32 at a time, and
// read the residual the same way: lanes that store rows of their own cost up to half of
// the time (16384 x 768 x 768 with a residual 34 us).  Tensor memory holds two sums, so that the epilogue
// runs beside the next unit's products.
//
// Tiles that do not fill the workers evenly are cut along the sum: worker p of P
// takes an equal share of all their steps, parts of a tile go to the
// workspace in fp32, and a second kernel adds a tile's parts in their order and
// runs the epilogue.
//
// What bounds it: with long sums the matrix unit and the card's power (16384 x 2048 x 8192
// with a residual 300 us, 1830 TFLOP/s, 97% of cuBLAS's burst; 350 where it runs on and
// on; the pipe busy in 87% of the cycles).  With a sum of 1024 the epilogue beside it: the
// products alone take 71 us for 16384 x 4096, with the stores 87, with GELU 97, with z
// stored too 108 (57% of the cycles); shared memory, which feeds the products at half its
// rate, also carries the stores.  Small products: copies, 64 bytes a clock into an SM (a
// step of 32 KB 0.27 us), after 5 us for a tile's start and end (128 x 128 x 64; 777 x
// 1301 x 1001 at odd starts 16 us with the copies that align it).
#include <type_traits>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

__device__ unsigned g_linear_error;

constexpr int BK = 64;            // of the sum a step
constexpr int kEpWarps = 16;
constexpr int kGroup = 32;        // columns of a warp's 32 rows that it stores at a time
constexpr uint32_t kBuf = 32 * kGroup * 2;  // bytes of them; a warp has two, or one in fp32
constexpr int kGemmThreads = 64 + 32 * kEpWarps;

template <int CG>
struct Shape {
  static constexpr int kRows = 128 * CG;       // of a tile
  static constexpr int kCols = 128 * CG;
  static constexpr int kStages = 5;
  static constexpr uint32_t kA = 128 * BK * 2, kB = 128 * BK * 2, kStage = kA + kB;
  static constexpr uint32_t kAlloc = 2 * kCols;  // columns of tensor memory
  static constexpr uint32_t kArea = kStages * kStage;  // offset of the warps' own areas
  static constexpr uint32_t kBytes = 1024 + kArea + kEpWarps * 2 * kBuf;
};
static_assert(Shape<2>::kBytes <= 226 * 1024, "with the barriers, an SM's 227 KB");

struct GemmArgs {
  CUtensorMap a, b, out, z, residual;  // the last three where ep.tiled and there is one
  int a_mn, b_mn;
  int64_t M, N;
  int steps;             // of the sum
  int tiles_m, tiles_n;
  int whole;             // tiles that one worker takes whole; the others are cut
  int workers;
  uint32_t shape;
  uint32_t stage;        // bytes of a step's copies to a block
  Epilogue ep;
  float* partial;        // [worker][2][rows][cols]
  __device__ __forceinline__ bool second(unsigned) const { return false; }
  __device__ __forceinline__ const GemmArgs& of(bool) const { return *this; }
  __device__ __forceinline__ int from(bool) const { return 0; }
};

// One product, or two that together leave no block without one: those from `first` on work
// at the second.
struct GemmPair {
  GemmArgs g[2];
  int first;
  __device__ __forceinline__ bool second(unsigned block) const { return (int)block >= first; }
  __device__ __forceinline__ const GemmArgs& of(bool second) const { return g[second]; }
  __device__ __forceinline__ int from(bool second) const { return second ? first : 0; }
};

// Tile t in an order in which tiles that run at one time share operands: strips
// of eight tile rows, column by column.
__host__ __device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int* tm,
                                                 int* tn) {
  const int strip = t / (8 * tiles_n), in = t - strip * (8 * tiles_n);
  const int high = tiles_m - 8 * strip < 8 ? tiles_m - 8 * strip : 8;
  *tn = in / high;
  *tm = 8 * strip + (in - *tn * high);
}

// First step of worker p's share of the cut tiles' `total` steps.
__host__ __device__ __forceinline__ int64_t share(int64_t total, int p, int workers) {
  return total * p / workers;
}

// A worker's units one after another: whole tiles, then its share.
struct Units {
  int i, p;
  int64_t at, end;
  int tile, k0, k1;  // the unit
  bool part;         // of a tile that others share
  int slot;
  __device__ __forceinline__ Units(const GemmArgs& a, int worker) : i(worker), p(worker) {
    const int64_t total = (int64_t)(a.tiles_m * a.tiles_n - a.whole) * a.steps;
    at = share(total, p, a.workers);
    end = share(total, p + 1, a.workers);
    slot = 0;
  }
  __device__ __forceinline__ bool next(const GemmArgs& a) {
    if (i < a.whole) {
      tile = i;
      i += a.workers;
      k0 = 0;
      k1 = a.steps;
      part = false;
      return true;
    }
    if (at >= end) return false;
    const int t = (int)(at / a.steps);
    const int64_t base = (int64_t)t * a.steps;
    tile = a.whole + t;
    k0 = (int)(at - base);
    k1 = end - base < a.steps ? (int)(end - base) : a.steps;
    part = k0 > 0 || k1 < a.steps;
    slot = k0 > 0 ? 0 : 1;  // a share's first tile may begin inside, its last end inside
    at = base + k1;
    return true;
  }
};

// ---------------------------------------------------------------------------
// Epilogue of a warp's 32 rows and 32 columns, a row a lane, sixteen columns at a time.
// ---------------------------------------------------------------------------

// Where 16-byte piece c (0..3) of a row of 64 bytes lies: as TMA's 64-byte swizzle has it, and
// the pieces of a warp's rows in different banks.
__device__ __forceinline__ uint4* piece(uint8_t* buf, int row, int c) {
  return reinterpret_cast<uint4*>(buf + row * 64 + ((c ^ (row >> 1 & 3)) << 4));
}
template <typename T>
__device__ __forceinline__ void put16(uint8_t* buf, int row, int half, const float (&z)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q)
    *piece(buf, row, 2 * half + q) =
        make_uint4(pack2<T>(z[8 * q], z[8 * q + 1]), pack2<T>(z[8 * q + 2], z[8 * q + 3]),
                   pack2<T>(z[8 * q + 4], z[8 * q + 5]), pack2<T>(z[8 * q + 6], z[8 * q + 7]));
}
template <typename T>
__device__ __forceinline__ void add16(const uint4& x, const uint4& y, float (&z)[16]) {
  const uint32_t o[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = unpack2<T>(o[k]);
    z[2 * k] += f.x;
    z[2 * k + 1] += f.y;
  }
}

// Tiled: columns n0 + 16 half .. of the group, into the buffers of z and y; the latter
// holds the residual.
template <typename T>
__device__ __forceinline__ void finish16(const Epilogue& e, float (&z)[16], int64_t n, int64_t N,
                                         int half, uint8_t* zbuf, uint8_t* ybuf) {
  const int lane = threadIdx.x & 31;
  if (e.bias) {
    const T* b = static_cast<const T*>(e.bias) + n;
    if (n + 16 <= N) {
      add16<T>(reinterpret_cast<const uint4*>(b)[0], reinterpret_cast<const uint4*>(b)[1], z);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (n + k < N) z[k] += to_f32(b[k]);
    }
  }
  if (e.z.data) put16<T>(zbuf, lane, half, z);
  by_act(e.act, [&](auto act) {
#pragma unroll
    for (int k = 0; k < 16; k += 2) act_of2<decltype(act)::value>(z[k], z[k + 1]);
  });
  if (e.residual.data) add16<T>(*piece(ybuf, lane, 2 * half), *piece(ybuf, lane, 2 * half + 1), z);
  put16<T>(ybuf, lane, half, z);
}

// At any alignment: the group has been put into `turn` in fp32 (turned), and a lane takes a
// column, row by row.
__device__ __forceinline__ float4* turned(float* turn, int row, int c) {  // piece c of 8 of a row
  return reinterpret_cast<float4*>(turn + row * 32 + ((c ^ (row & 7)) << 2));
}
__device__ __forceinline__ void put_turned(float* turn, int half, const float (&z)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *turned(turn, lane, 4 * half + q) = make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
}
template <typename T>
__device__ __forceinline__ void finish_turned(const Epilogue& e, const float* turn, int64_t m0,
                                              int64_t n0, int64_t M, int64_t N) {
  const int lane = threadIdx.x & 31;
  const int64_t n = n0 + lane;
  if (n >= N) return;
  const float bias = e.bias ? to_f32(static_cast<const T*>(e.bias)[n]) : 0.0f;
#pragma unroll 1
  for (int r0 = 0; r0 < 32 && m0 + r0 < M; r0 += 16) {
    T residual[16];  // sixteen rows' loads at once
    if (e.residual.data)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (m0 + r0 + r < M)
          residual[r] = static_cast<const T*>(e.residual.data)[(m0 + r0 + r) * e.residual.ld + n];
    by_act(e.act, [&](auto act) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = r0 + r;
        if (m0 + row >= M) break;
        const float v = turn[row * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
        const float x = e.bias ? v + bias : v;
        if (e.z.data) static_cast<T*>(e.z.data)[(m0 + row) * e.z.ld + n] = from_f32<T>(x);
        float y = act_of<decltype(act)::value>(x);
        if (e.residual.data) y += to_f32(residual[r]);
        static_cast<T*>(e.out.data)[(m0 + row) * e.out.ld + n] = from_f32<T>(y);
      }
    });
  }
}

// Whether the group of columns from n on is stored by TMA, which writes whole pieces of 16
// bytes: the last ones may have to end inside one.
__device__ __forceinline__ bool tiled_at(const GemmArgs& a, int64_t n) {
  return a.ep.tiled && (n + kGroup <= a.N || a.N % 8 == 0);
}

// What a warp of the epilogue keeps: two buffers of 32 x 32, and a barrier for each, on which
// the residual's bytes are counted.
struct Out {
  uint8_t* buf;
  uint64_t* bar;
  uint32_t par;  // bit b: of buffer b's next phase

  // Buffer of a group's y; z, if there is one, has the other.
  __device__ __forceinline__ int of(const Epilogue& e, int g) const { return e.z.data ? 1 : g & 1; }
  // By lane 0: both buffers are free.
  __device__ __forceinline__ void load(const GemmArgs& a, int b, int64_t m0, int64_t n0) {
    mbar_arrive_expect_tx(&bar[b], kBuf);
    tma_load2(buf + b * kBuf, &a.residual, (int)n0, (int)m0, &bar[b]);
  }
  // A wait ran out: lets loads that may be on their way land before the block ends.
  __device__ __forceinline__ void drain(const Epilogue& e) {
    for (int b = 0; e.residual.data && b < 2; ++b)
      mbar_wait(&bar[b], par >> b & 1, &g_linear_error, kErrDrain);
  }
  // Before a unit's (parts of) GROUPS groups from (m0, n0) on: the buffers' last stores have
  // been read, and the residual is on its way.
  template <int GROUPS>
  __device__ __forceinline__ void begin(const GemmArgs& a, int64_t m0, int64_t n0) {
    if ((threadIdx.x & 31) == 0) {
      store_wait_read<0>();
      if (a.ep.residual.data && m0 < a.M)
        for (int g = 0; g < (a.ep.z.data ? 1 : GROUPS); ++g)
          if (n0 + g * kGroup < a.N && tiled_at(a, n0 + g * kGroup))
            load(a, of(a.ep, g), m0, n0 + g * kGroup);
    }
    __syncwarp();
  }
  // Group g, whose sums come by get(half, z); whole warps, inside the matrix.
  template <typename T, typename F>
  __device__ __forceinline__ bool group(const GemmArgs& a, int g, int64_t m0, int64_t n0, F get) {
    const Epilogue& e = a.ep;
    const int lane = threadIdx.x & 31, b = of(e, g);
    uint8_t *ybuf = buf + b * kBuf, *zbuf = buf;
    if (e.z.data && g > 0) {  // one pair of buffers for all groups
      if (lane == 0) {
        store_wait_read<0>();
        if (e.residual.data) load(a, b, m0, n0);
      }
      __syncwarp();
    }
    if (e.residual.data) {
      if (!warp_wait(&bar[b], par >> b & 1, &g_linear_error)) return false;
      par ^= 1u << b;
    }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      float z[16];
      get(half, z);
      finish16<T>(e, z, n0 + 16 * half, a.N, half, zbuf, ybuf);
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (e.z.data) tma_store2(&a.z, (int)n0, (int)m0, zbuf);
      tma_store2(&a.out, (int)n0, (int)m0, ybuf);
      store_commit();
    }
    return true;
  }
};

// Sums of 32 rows and 16 columns in the workspace: four columns of a lane side by side, the
// lanes' behind one another.
__device__ __forceinline__ float4* part_at(float* partial, int64_t slot, int rows, int cols, int row0,
                                           int c) {
  return reinterpret_cast<float4*>(partial + slot * rows * cols + (int64_t)row0 * cols + c * 32) +
         (threadIdx.x & 31);
}

struct GemmBars {
  uint64_t full[8], empty[8], sum_full[2], sum_empty[2], drain, residual[kEpWarps][2];
  uint32_t tmem;
};

// Args: GemmArgs, or GemmPair.
template <int CG, typename Args>
__global__ void __launch_bounds__(kGemmThreads, 1) k_gemm(const __grid_constant__ Args args) {
  using S = Shape<CG>;
  const bool second = args.second(blockIdx.x);
  const GemmArgs& a = args.of(second);
  extern __shared__ uint8_t raw[];
  __shared__ GemmBars bar;
  uint8_t* smem = align_shared(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int worker = ((int)blockIdx.x - args.from(second)) / CG;

  if (threadIdx.x == 0) {
    map_prefetch(&a.a);
    map_prefetch(&a.b);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.sum_full[i], 1);
      mbar_init(&bar.sum_empty[i], kEpWarps * CG);
    }
    mbar_init(&bar.drain, 1);
    for (int i = 0; i < 2 * kEpWarps; ++i) mbar_init(&bar.residual[0][0] + i, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    if (CG == 2)
      pair_alloc(&bar.tmem, S::kAlloc);
    else
      tmem_alloc(&bar.tmem, S::kAlloc);
  }
  tc_fence_before();
  if (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  grid_wait();

  // Steps of this worker in all: what nobody waits for is not signalled.
  int64_t mine = 0;
  if (warp <= 1) {
    Units u(a, worker);
    while (u.next(a)) mine += u.k1 - u.k0;
  }

  if (warp == 0) {
    // ----- copies ----------------------------------------------------------
    Units u(a, worker);
    bool ok = true;
    int st = 0, par = 1;
    int64_t n = 0;  // steps asked for
    while (ok && u.next(a)) {
      int tm, tn;
      tile_at(u.tile, a.tiles_m, a.tiles_n, &tm, &tn);
      const int m0 = tm * S::kRows + (int)rank * 128, n0 = tn * S::kCols + (int)rank * 128 * (CG - 1);
      for (int k = u.k0; k < u.k1; ++k) {
        if (n >= S::kStages) ok = warp_wait(&bar.empty[st], par, &g_linear_error, kErrWaitEmpty);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* to = smem + st * S::kStage;
          if (CG == 2) {
            const uint32_t full = cluster_addr(smem_u32(&bar.full[st]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&bar.full[st], 2 * a.stage);
            if (a.a_mn) {
              pair_load2(to, &a.a, m0, k * BK, full);
              pair_load2(to + S::kA / 2, &a.a, m0 + 64, k * BK, full);
            } else {
              pair_load2(to, &a.a, k * BK, m0, full);
            }
            if (a.b_mn) {
              pair_load2(to + S::kA, &a.b, n0, k * BK, full);
              pair_load2(to + S::kA + S::kB / 2, &a.b, n0 + 64, k * BK, full);
            } else {
              pair_load2(to + S::kA, &a.b, k * BK, n0, full);
            }
          } else {
            mbar_arrive_expect_tx(&bar.full[st], a.stage);
            if (a.a_mn) {
              tma_load2(to, &a.a, m0, k * BK, &bar.full[st]);
              tma_load2(to + S::kA / 2, &a.a, m0 + 64, k * BK, &bar.full[st]);
            } else {
              tma_load2(to, &a.a, k * BK, m0, &bar.full[st]);
            }
            if (a.b_mn) {
              tma_load2(to + S::kA, &a.b, n0, k * BK, &bar.full[st]);
              tma_load2(to + S::kA + S::kB / 2, &a.b, n0 + 64, k * BK, &bar.full[st]);
            } else {
              tma_load2(to + S::kA, &a.b, k * BK, n0, &bar.full[st]);
            }
          }
        }
        ++n;
        if (++st == S::kStages) st = 0, par ^= 1;
      }
    }
    if (!ok && rank == 0)  // a wait ran out: let what is in flight land before the block ends
      for (int64_t i = n > S::kStages ? n - S::kStages : 0; i < n; ++i)
        mbar_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1, &g_linear_error, kErrDrain);
  } else if (warp == 1) {
    // ----- products --------------------------------------------------------
    if (rank == 0) {
      const uint32_t leader = elect_lane();
      const uint32_t base = smem_u32(smem);
      const uint64_t a_desc = a.a_mn ? desc_mn(base, S::kA / 2) : desc_k(base);
      const uint64_t b_desc = a.b_mn ? desc_mn(base + S::kA, S::kB / 2) : desc_k(base + S::kA);
      const uint32_t a_step = (a.a_mn ? 2048 : 32) >> 4, b_step = (a.b_mn ? 2048 : 32) >> 4;
      Units u(a, worker);
      bool ok = true;
      int st = 0, par = 0, buf = 0, sum_par = 1;
      int64_t n = 0;
      int64_t units = 0;
      while (ok && u.next(a)) {
        if (units >= 2) ok = warp_wait(&bar.sum_empty[buf], sum_par, &g_linear_error, kErrWaitEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * S::kCols;
        for (int k = u.k0; k < u.k1; ++k) {
          ok = warp_wait(&bar.full[st], par, &g_linear_error);
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = a_desc + (uint32_t)st * (S::kStage >> 4);
          const uint64_t bd = b_desc + (uint32_t)st * (S::kStage >> 4);
#pragma unroll
          for (int s = 0; s < BK / 16; ++s) {
            const bool add = k > u.k0 || s > 0;
            if (CG == 2)
              pair_mma(leader, d, ad + s * a_step, bd + s * b_step, a.shape, add);
            else
              mma_ss(leader, d, ad + s * a_step, bd + s * b_step, a.shape, add);
          }
          // Only where a later copy waits for it: nothing may arrive after the block's end.
          if (n + S::kStages < mine) {
            if (CG == 2)
              pair_commit(leader, &bar.empty[st]);
            else
              mma_commit(leader, &bar.empty[st]);
          }
          ++n;
          if (++st == S::kStages) st = 0, par ^= 1;
        }
        if (!ok) break;
        if (CG == 2)
          pair_commit(leader, &bar.sum_full[buf]);
        else
          mma_commit(leader, &bar.sum_full[buf]);
        ++units;
        if (++buf == 2) buf = 0, sum_par ^= 1;
      }
      if (!ok) {
        // the copies, which were asked for as far as the stages go, and the products
        for (int64_t i = n; i < n + S::kStages && i < mine; ++i)
          mbar_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1, &g_linear_error, kErrDrain);
        if (CG == 2)  // the other block waits for no such arrival, and may have ended
          pair_commit_here(leader, &bar.drain);
        else
          mma_commit(leader, &bar.drain);
        mbar_wait(&bar.drain, 0, &g_linear_error, kErrDrain);
      }
    }
  } else {
    // ----- epilogue --------------------------------------------------------
    // A warp reaches 32 lanes of tensor memory, by its number; four share them, a quarter
    // of the columns each.
    constexpr int kCols = S::kCols / (kEpWarps / 4);
    const int w = warp - 2, lanes0 = (warp & 3) * 32, col0 = (w >> 2) * kCols;
    Out out{smem + S::kArea + w * 2 * kBuf, bar.residual[w], 0};
    float* turn = reinterpret_cast<float*>(out.buf);
    const uint32_t lanes = (uint32_t)lanes0 << 16;
    const uint32_t empty = CG == 2 ? cluster_addr(smem_u32(&bar.sum_empty[0]), 0) : 0;
    Units u(a, worker);
    bool ok = true;
    int buf = 0, par = 0;
    while (ok && u.next(a)) {
      int tm, tn;
      tile_at(u.tile, a.tiles_m, a.tiles_n, &tm, &tn);
      const int row0 = (int)rank * 128 + lanes0;  // in the tile
      const int64_t m0 = (int64_t)tm * S::kRows + row0, n0 = (int64_t)tn * S::kCols + col0;
      if (a.ep.tiled && !u.part) out.begin<kCols / kGroup>(a, m0, n0);
      ok = warp_wait(&bar.sum_full[buf], par, &g_linear_error);
      if (!ok) break;
      tc_fence_after();
      int taken = 0;  // columns
      auto get = [&](int, float (&z)[16]) {
        uint32_t r[16];
        __syncwarp();  // one lane may come from a copy of its own
        tmem_ld16(r, tmem + lanes + buf * S::kCols + col0 + taken);
        tmem_wait_ld(r);
        taken += 16;
#pragma unroll
        for (int k = 0; k < 16; ++k) z[k] = __uint_as_float(r[k]);
        if (taken < kCols) return;
        tc_fence_before();  // the last: the next sum may come
        __syncwarp();
        if (lane == 0) {
          if (CG == 2)
            cluster_arrive(empty + 8 * buf);
          else
            mbar_arrive(&bar.sum_empty[buf]);
        }
      };
#pragma unroll 1
      for (int g = 0; ok && g < kCols / kGroup; ++g) {
        const int64_t n = n0 + g * kGroup;
        const bool inside = m0 < a.M && n < a.N;
        if (u.part || !inside || !tiled_at(a, n)) {
          if (lane == 0) store_wait_read<0>();
          __syncwarp();  // the groups before have been read
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            float z[16];
            get(half, z);
            if (u.part && m0 < a.M) {
              float4* p = part_at(a.partial, (int64_t)worker * 2 + u.slot, S::kRows, S::kCols, row0,
                                  col0 + g * kGroup + 16 * half);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                p[32 * q] = make_float4(z[4 * q], z[4 * q + 1], z[4 * q + 2], z[4 * q + 3]);
            } else if (!u.part && inside) {
              put_turned(turn, half, z);
            }
          }
          if (u.part || !inside) continue;
          __syncwarp();
          if (a.ep.type == OB_TYPE_BF16)
            finish_turned<__nv_bfloat16>(a.ep, turn, m0, n, a.M, a.N);
          else
            finish_turned<__half>(a.ep, turn, m0, n, a.M, a.N);
        } else if (a.ep.type == OB_TYPE_BF16) {
          ok = out.group<__nv_bfloat16>(a, g, m0, n, get);
        } else {
          ok = out.group<__half>(a, g, m0, n, get);
        }
      }
      __syncwarp();
      if (++buf == 2) buf = 0, par ^= 1;
    }
    if (!ok) out.drain(a.ep);
    if (lane == 0) store_wait_read<0>();
    __syncwarp();
    tc_fence_before();
  }
  if (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (CG == 2)
      pair_free(tmem, S::kAlloc);
    else
      tmem_free(tmem, S::kAlloc);
  }
}

// The cut tiles: a warp 32 rows of 32 columns, its parts in their order.
template <int CG>
__global__ void __launch_bounds__(256) k_gemm_parts(const __grid_constant__ GemmArgs a) {
  using S = Shape<CG>;
  __shared__ __align__(1024) uint8_t bufs[8][2 * kBuf];
  __shared__ uint64_t bars[8][2];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    mbar_init(&bars[w][0], 1);
    mbar_init(&bars[w][1], 1);
    fence_barrier_init();
  }
  __syncwarp();
  grid_wait();
  constexpr int kAcross = S::kCols / kGroup, kPer = (S::kRows / 32) * kAcross;  // warps a tile
  const int unit = blockIdx.x * 8 + w, t = unit / kPer, in = unit % kPer;
  const int row0 = in / kAcross * 32, c = in % kAcross * kGroup;
  int tm, tn;
  tile_at(a.whole + t, a.tiles_m, a.tiles_n, &tm, &tn);
  const int64_t m0 = (int64_t)tm * S::kRows + row0, n0 = (int64_t)tn * S::kCols + c;
  if (m0 >= a.M || n0 >= a.N) return;
  const int64_t total = (int64_t)(a.tiles_m * a.tiles_n - a.whole) * a.steps;
  const int64_t first = (int64_t)t * a.steps, last = first + a.steps - 1;
  // the worker of a step: the largest p with share(p) <= step
  auto owner = [&](int64_t step) {
    int p = (int)(step * a.workers / total);
    while (p + 1 < a.workers && share(total, p + 1, a.workers) <= step) ++p;
    while (share(total, p, a.workers) > step) --p;
    return p;
  };
  int p0 = 0, p1 = -1;
  if (total > 0) {  // else the sums are empty
    p0 = owner(first);
    p1 = owner(last);
    if (p0 == p1) return;  // one worker had it whole
  }
  Out out{bufs[w], bars[w], 0};
  auto get = [&](int half, float (&z)[16]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) z[k] = 0.0f;
    // Every worker between has a step; the first alone may have begun before this tile.
    constexpr int B = 4;  // parts on their way at once
    for (int p = p0; p <= p1; p += B) {
      float4 v[B][4];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (p + b > p1) break;
        const int slot = p + b == p0 && share(total, p0, a.workers) <= first ? 1 : 0;
        const float4* q =
            part_at(a.partial, (int64_t)(p + b) * 2 + slot, S::kRows, S::kCols, row0, c + 16 * half);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[b][k] = q[32 * k];
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (p + b > p1) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z[4 * k] += v[b][k].x;
          z[4 * k + 1] += v[b][k].y;
          z[4 * k + 2] += v[b][k].z;
          z[4 * k + 3] += v[b][k].w;
        }
      }
    }
  };
  if (tiled_at(a, n0)) {
    out.begin<1>(a, m0, n0);
    const bool ok = a.ep.type == OB_TYPE_BF16 ? out.group<__nv_bfloat16>(a, 0, m0, n0, get)
                                              : out.group<__half>(a, 0, m0, n0, get);
    if (!ok) out.drain(a.ep);
    if (lane == 0) store_wait_read<0>();
    return;
  }
  float* turn = reinterpret_cast<float*>(out.buf);
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    float z[16];
    get(half, z);
    put_turned(turn, half, z);
  }
  __syncwarp();
  if (a.ep.type == OB_TYPE_BF16)
    finish_turned<__nv_bfloat16>(a.ep, turn, m0, n0, a.M, a.N);
  else
    finish_turned<__half>(a.ep, turn, m0, n0, a.M, a.N);
}

constexpr int kSms = 152;

struct Plan {
  int cg, tiles_m, tiles_n, steps, workers, whole;
};

// Rows of A that a block copies: few rows are copied as they are, and what the other rows of
// the tile hold gives sums that nobody reads.
int copied_rows(int64_t M, bool a_mn) { return M < 128 && !a_mn ? (int)((M + 7) / 8 * 8) : 128; }

// What a product is cut into.  By sizes and a_mn alone: the workspace goes by it.
Plan plan_of(int64_t M, int64_t N, int64_t K, bool a_mn) {
  const int64_t steps = (K + BK - 1) / BK;
  // A step takes about 0.27 us in either form: a block's copies of 32 KB, which a pair needs
  // for four times the products.  Cutting the last tiles costs the second kernel and its
  // traffic, about 4.5 us (16 steps); a pair's epilogue is the longer one.
  auto form = [&](int cg, int64_t* time) {
    Plan p{};
    p.cg = cg;
    const int edge = 128 * cg, most = kSms / cg;
    p.tiles_m = (int)((M + edge - 1) / edge);
    p.tiles_n = (int)((N + edge - 1) / edge);
    p.steps = (int)steps;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, rest = tiles % most;
    const int64_t cost = cg == 1 ? 16 * 256 / (copied_rows(M, a_mn) + 128) : 16;
    p.workers = (int)(tiles < most ? tiles : most);
    p.whole = steps ? (int)tiles : 0;
    *time = (tiles + most - 1) / most * steps + 4 * cg;
    // A worker has four steps at least (the others' parts of a tile are summed as if every
    // one between had some), or the parts are more than their sum is worth.
    int64_t workers = most;
    if (rest == tiles && rest * steps / 4 < most) workers = rest * steps / 4;
    if (rest && workers > rest && rest * steps >= 4 * workers) {
      const int64_t share = (rest * steps + workers - 1) / workers;
      if (steps - share > cost) {
        p.whole = (int)(tiles - rest);
        p.workers = (int)workers;
        *time = tiles / most * steps + share + cost + 4 * cg;
      }
    }
    return p;
  };
  int64_t t1, t2;
  const Plan p1 = form(1, &t1), p2 = form(2, &t2);
  return t2 < t1 ? p2 : p1;
}

template <int CG>
cudaError_t fill(const Gemm& g, const Plan& p, GemmArgs* out) {
  using S = Shape<CG>;
  GemmArgs& a = *out;
  cudaError_t e = cudaSuccess;
  auto map = [&](CUtensorMap* to, const Mat& m, int64_t rows, int64_t cols, int bc, int br) {
    if (e == cudaSuccess) e = matrix_tensor_map(to, m, g.ep.type, rows, cols, bc, br);
  };
  const int a_rows = CG == 1 ? copied_rows(g.M, g.a_mn) : 128;
  a.stage = a_rows * BK * 2 + S::kB;
  if (p.steps) {
    if (g.a_mn)
      map(&a.a, g.a, g.K, g.M, 64, BK);
    else
      map(&a.a, g.a, g.M, g.K, 64, a_rows);
    if (g.b_mn)
      map(&a.b, g.b, g.K, g.N, 64, BK);
    else
      map(&a.b, g.b, g.N, g.K, 64, 128);
  }
  if (g.ep.tiled) {
    map(&a.out, g.ep.out, g.M, g.N, kGroup, 32);
    if (g.ep.z.data) map(&a.z, g.ep.z, g.M, g.N, kGroup, 32);
    if (g.ep.residual.data) map(&a.residual, g.ep.residual, g.M, g.N, kGroup, 32);
  }
  a.a_mn = g.a_mn;
  a.b_mn = g.b_mn;
  a.M = g.M;
  a.N = g.N;
  a.steps = p.steps;
  a.tiles_m = p.tiles_m;
  a.tiles_n = p.tiles_n;
  a.whole = p.whole;
  a.workers = p.workers;
  a.shape = mma_shape(g.ep.type == OB_TYPE_BF16, S::kCols, g.b_mn, g.a_mn, S::kRows);
  a.ep = g.ep;
  a.partial = g.partial;
  return e;
}

template <int CG, typename Args>
cudaError_t run_products(const Args& args, int blocks, cudaStream_t s) {
  using S = Shape<CG>;
  static PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_gemm<CG, Args>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)S::kBytes);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(kGemmThreads);
  c.dynamicSmemBytes = S::kBytes;
  c.stream = s;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = CG;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&c, k_gemm<CG, Args>, args);
}
// The second kernel of a product that is cut.
template <int CG>
cudaError_t run_parts(const GemmArgs& a, cudaStream_t s) {
  using S = Shape<CG>;
  const int rest = a.tiles_m * a.tiles_n - a.whole;
  if (!rest) return cudaSuccess;
  return launch_behind(k_gemm_parts<CG>, dim3(rest * ((S::kRows / 32) * (S::kCols / kGroup) / 8)),
                       dim3(256), 0, s, a);
}

template <int CG>
cudaError_t run_one(const Gemm& g, const Plan& p, cudaStream_t s) {
  GemmArgs a{};
  cudaError_t e = fill<CG>(g, p, &a);
  if (e == cudaSuccess && p.steps) e = run_products<CG>(a, a.workers * CG, s);
  return e == cudaSuccess ? run_parts<CG>(a, s) : e;
}

}  // namespace

size_t gemm_partial_bytes(int64_t M, int64_t N, int64_t K, bool a_mn, bool pair) {
  if (M == 0 || N == 0) return 0;
  if (few_rows(M, N, K, a_mn, pair)) return 0;
  const Plan p = plan_of(M, N, K, a_mn);
  if (p.whole == p.tiles_m * p.tiles_n || !p.steps) return 0;
  return (size_t)p.workers * 2 * (128 * p.cg) * (128 * p.cg) * sizeof(float);
}

cudaError_t launch_gemm(const Gemm& g, cudaStream_t s) {
  if (g.M == 0 || g.N == 0) return cudaSuccess;
  if (few_rows(g.M, g.N, g.K, g.a_mn, g.pair)) return launch_few(g, s);
  const Plan p = plan_of(g.M, g.N, g.K, g.a_mn);
  return p.cg == 2 ? run_one<2>(g, p, s) : run_one<1>(g, p, s);
}

cudaError_t launch_gemms(const Gemm& g, const Gemm& h, cudaStream_t s) {
  auto tiled = [](const Gemm& p) { return p.M > 0 && p.N > 0 && !few_rows(p.M, p.N, p.K, p.a_mn, p.pair); };
  const bool both = tiled(g) && tiled(h);
  if (both) {
    const Plan p = plan_of(g.M, g.N, g.K, g.a_mn), q = plan_of(h.M, h.N, h.K, h.a_mn);
    if (p.cg == 1 && q.cg == 1 && p.steps && q.steps && p.workers + q.workers <= kSms) {
      GemmPair pair{};
      pair.first = p.workers;
      cudaError_t e = fill<1>(g, p, &pair.g[0]);
      if (e == cudaSuccess) e = fill<1>(h, q, &pair.g[1]);
      if (e == cudaSuccess) e = run_products<1>(pair, p.workers + q.workers, s);
      if (e == cudaSuccess) e = run_parts<1>(pair.g[0], s);
      return e == cudaSuccess ? run_parts<1>(pair.g[1], s) : e;
    }
  }
  const cudaError_t e = launch_gemm(g, s);
  return e == cudaSuccess ? launch_gemm(h, s) : e;
}

cudaError_t linear_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_linear_error);
}

}  // namespace ob
