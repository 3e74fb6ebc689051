// One product of the dense layer on the tensor cores, with its epilogue.
//
// Workers stay and take unit after unit of the output: a pair of blocks a tile
// of 256 x 256 (each holds 128 rows of A and of the sum, and half of B), or, where
// that leaves most of the card idle, a block a tile of 128 x 128.  In a block one
// warp issues the copies (tiles of 64 along the sum, 128-byte swizzle, either
// operand stored along the sum or across it), one the products, and sixteen
// take the sums out of tensor memory, 16 columns of a row a thread: bias,
// activation, residual, one rounding.  Tensor memory holds two sums, so that the epilogue
// runs beside the next unit's products.
//
// Tiles that do not fill the workers evenly are cut along the sum: worker p of P
// takes an equal share of all their steps, parts of a tile go to the
// workspace in fp32, and a second kernel adds a tile's parts in their order and
// runs the epilogue.
#include <atomic>
#include <type_traits>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

__device__ unsigned g_layer_error;

constexpr int BK = 64;            // of the sum a step
constexpr int kEpWarps = 16;
constexpr int kEpCols = 16;       // columns of a row that a lane takes at a time
constexpr int kTurn = 16 * (kEpCols + 1);  // floats of a warp's own area: half of its rows
constexpr int kGemmThreads = 64 + 32 * kEpWarps;

template <int CG>
struct Shape {
  static constexpr int kRows = 128 * CG;       // of a tile
  static constexpr int kCols = 128 * CG;
  static constexpr int kStages = 6;
  static constexpr uint32_t kA = 128 * BK * 2, kB = 128 * BK * 2, kStage = kA + kB;
  static constexpr uint32_t kAlloc = 2 * kCols;  // columns of tensor memory
  static constexpr uint32_t kArea = kStages * kStage;  // offset of the warps' own areas
  static constexpr uint32_t kBytes = 1024 + kArea + kEpWarps * kTurn * 4;
};
static_assert(Shape<2>::kBytes <= 226 * 1024, "with the barriers, an SM's 227 KB");

struct GemmArgs {
  CUtensorMap a, b;
  int a_mn, b_mn;
  int64_t M, N;
  int steps;             // of the sum
  int tiles_m, tiles_n;
  int whole;             // tiles that one worker takes whole; the others are cut
  int workers;
  uint32_t shape;
  Epilogue ep;
  float* partial;        // [worker][2][rows][cols]
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

// Eight 4-byte words at once, or (`wide` 1) twice four where a row is only 16-byte aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t* v, int wide = 2) {
  if (wide == 1) {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void load32(const void* p, uint32_t* v, int wide = 2) {
  if (wide == 1) {
    const uint4 x = static_cast<const uint4*>(p)[0], y = static_cast<const uint4*>(p)[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    return;
  }
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
                 "=r"(v[7])
               : "l"(p)
               : "memory");
}

// z without bias -> outputs, for 16 columns from n on of row m, a row a lane.
template <typename T>
__device__ __forceinline__ void epilogue_wide(const Epilogue& e, float (&z)[kEpCols], int64_t m,
                                              int64_t n, bool row) {
  uint32_t o[8];
  if (e.bias) {
    const uint4* b = reinterpret_cast<const uint4*>(static_cast<const T*>(e.bias) + n);
    const uint4 x = b[0], y = b[1];
    o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
    o[4] = y.x, o[5] = y.y, o[6] = y.z, o[7] = y.w;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = unpack2<T>(o[k]);
      z[2 * k] += f.x;
      z[2 * k + 1] += f.y;
    }
  }
  if (e.z.data && row) {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = pack2<T>(z[2 * k], z[2 * k + 1]);
    store32(static_cast<T*>(e.z.data) + m * e.z.ld + n, o, e.wide);
  }
  if (e.residual.data && row)
    load32(static_cast<const T*>(e.residual.data) + m * e.residual.ld + n, o, e.wide);
  by_act(e.act, [&](auto act) {
#pragma unroll
    for (int k = 0; k < kEpCols; k += 2) act_of2<decltype(act)::value>(z[k], z[k + 1]);
  });
  if (e.residual.data)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 f = unpack2<T>(o[k]);
      z[2 * k] += f.x;
      z[2 * k + 1] += f.y;
    }
  if (!row) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = pack2<T>(z[2 * k], z[2 * k + 1]);
  store32(static_cast<T*>(e.out.data) + m * e.out.ld + n, o, e.wide);
}

// The same at any alignment and at the matrix's edges: turned through the
// warp's own shared memory, a column of every second row a lane.
template <typename T>
__device__ __forceinline__ void epilogue_edge(const Epilogue& e, const float (&z)[kEpCols],
                                              int64_t m0, int64_t n0, int64_t M, int64_t N,
                                              float* turn) {
  const int lane = threadIdx.x & 31, col = lane & (kEpCols - 1);
  const int64_t n = n0 + col;
  const float bias = e.bias && n < N ? to_f32(static_cast<const T*>(e.bias)[n]) : 0.0f;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
    if (lane / 16 == h)
#pragma unroll
      for (int k = 0; k < kEpCols; ++k) turn[lane % 16 * (kEpCols + 1) + k] = z[k];
    __syncwarp();
    if (n >= N) continue;
    const int64_t m = m0 + 16 * h;
    const int rows = M - m < 16 ? (int)(M - m) : 16;
    by_act(e.act, [&](auto act) {
#pragma unroll 4
      for (int r = lane / kEpCols; r < rows; r += 32 / kEpCols) {
        const float v = turn[r * (kEpCols + 1) + col], x = e.bias ? v + bias : v;
        if (e.z.data) static_cast<T*>(e.z.data)[(m + r) * e.z.ld + n] = from_f32<T>(x);
        float y = act_of<decltype(act)::value>(x);
        if (e.residual.data)
          y += to_f32(static_cast<const T*>(e.residual.data)[(m + r) * e.residual.ld + n]);
        static_cast<T*>(e.out.data)[(m + r) * e.out.ld + n] = from_f32<T>(y);
      }
    });
  }
}

// m0, n0: the warp's first row and column.
template <typename T>
__device__ __forceinline__ void epilogue(const Epilogue& e, float (&z)[kEpCols], int64_t m0,
                                         int64_t n0, int64_t M, int64_t N, float* turn) {
  if (n0 >= N || m0 >= M) return;
  const int64_t m = m0 + (threadIdx.x & 31);
  if (e.wide && n0 + kEpCols <= N)
    epilogue_wide<T>(e, z, m, n0, m < M);
  else
    epilogue_edge<T>(e, z, m0, n0, M, N, turn);
}

struct GemmBars {
  uint64_t full[8], empty[8], sum_full[2], sum_empty[2], drain;
  uint32_t tmem;
};

template <int CG>
__global__ void __launch_bounds__(kGemmThreads, 1) k_gemm(const __grid_constant__ GemmArgs a) {
  using S = Shape<CG>;
  extern __shared__ uint8_t raw[];
  __shared__ GemmBars bar;
  uint8_t* smem = align_shared(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  const int worker = blockIdx.x / CG;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.sum_full[i], 1);
      mbar_init(&bar.sum_empty[i], kEpWarps * CG);
    }
    mbar_init(&bar.drain, 1);
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
        if (n >= S::kStages) ok = warp_wait(&bar.empty[st], par, &g_layer_error, kErrWaitEmpty);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* to = smem + st * S::kStage;
          if (CG == 2) {
            const uint32_t full = cluster_addr(smem_u32(&bar.full[st]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&bar.full[st], 2 * S::kStage);
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
            mbar_arrive_expect_tx(&bar.full[st], S::kStage);
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
        mbar_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1, &g_layer_error, kErrDrain);
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
        if (units >= 2) ok = warp_wait(&bar.sum_empty[buf], sum_par, &g_layer_error, kErrWaitEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * S::kCols;
        for (int k = u.k0; k < u.k1; ++k) {
          ok = warp_wait(&bar.full[st], par, &g_layer_error);
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
        if (CG == 2)
          pair_commit(leader, &bar.drain);
        else
          mma_commit(leader, &bar.drain);
        mbar_wait(&bar.drain, 0, &g_layer_error, kErrDrain);
      }
    }
  } else {
    // ----- epilogue --------------------------------------------------------
    // A warp reaches 32 lanes of tensor memory, by its number; four share them, a quarter
    // of the columns each.
    constexpr int kCols = S::kCols / (kEpWarps / 4);
    const int w = warp - 2, lanes0 = (warp & 3) * 32, col0 = (w >> 2) * kCols;
    float* turn = reinterpret_cast<float*>(smem + S::kArea) + w * kTurn;
    const uint32_t lanes = (uint32_t)lanes0 << 16;
    const uint32_t empty = CG == 2 ? cluster_addr(smem_u32(&bar.sum_empty[0]), 0) : 0;
    Units u(a, worker);
    bool ok = true;
    int buf = 0, par = 0;
    while (ok && u.next(a)) {
      ok = warp_wait(&bar.sum_full[buf], par, &g_layer_error);
      if (!ok) break;
      tc_fence_after();
      int tm, tn;
      tile_at(u.tile, a.tiles_m, a.tiles_n, &tm, &tn);
      const int row0 = (int)rank * 128 + lanes0;  // in the tile
      const int64_t m0 = (int64_t)tm * S::kRows + row0;
#pragma unroll 1
      for (int c = col0; c < col0 + kCols; c += kEpCols) {
        uint32_t r[kEpCols];
        __syncwarp();  // the last columns' lanes may have parted at an edge
        tmem_ld16(r, tmem + lanes + buf * S::kCols + c);
        tmem_wait_ld(r);
        if (c + kEpCols == col0 + kCols) {  // the last: the next sum may come
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2)
              cluster_arrive(empty + 8 * buf);
            else
              mbar_arrive(&bar.sum_empty[buf]);
          }
        }
        if (u.part) {
          float* p = a.partial + (((int64_t)worker * 2 + u.slot) * S::kRows + row0 + lane) * S::kCols + c;
          store32(p, r);
          store32(p + 8, r + 8);
        } else {
          float z[kEpCols];
#pragma unroll
          for (int k = 0; k < kEpCols; ++k) z[k] = __uint_as_float(r[k]);
          const int64_t n0 = (int64_t)tn * S::kCols + c;
          if (a.ep.type == OB_TYPE_BF16)
            epilogue<__nv_bfloat16>(a.ep, z, m0, n0, a.M, a.N, turn);
          else
            epilogue<__half>(a.ep, z, m0, n0, a.M, a.N, turn);
        }
      }
      if (++buf == 2) buf = 0, par ^= 1;
    }
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

// The cut tiles: a warp 32 rows of 16 columns, its parts in their order.
template <int CG>
__global__ void __launch_bounds__(256) k_gemm_parts(const __grid_constant__ GemmArgs a) {
  using S = Shape<CG>;
  __shared__ float turn[8][kTurn];
  grid_wait();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kAcross = S::kCols / kEpCols, kPer = (S::kRows / 32) * kAcross;  // warps a tile
  const int unit = blockIdx.x * 8 + w, t = unit / kPer, in = unit % kPer;
  const int row0 = in / kAcross * 32, c = in % kAcross * kEpCols;
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
  float z[kEpCols];
#pragma unroll
  for (int k = 0; k < kEpCols; ++k) z[k] = 0.0f;
  int p0 = 0, p1 = -1;
  if (total > 0) {  // else the sums are empty
    p0 = owner(first);
    p1 = owner(last);
    if (p0 == p1) return;  // one worker had it whole
  }
  for (int p = p0; p <= p1; ++p) {
    if (share(total, p, a.workers) == share(total, p + 1, a.workers)) continue;  // no step at all
    const int slot = share(total, p, a.workers) > first ? 0 : 1;
    const float* q =
        a.partial + (((int64_t)p * 2 + slot) * S::kRows + row0 + lane) * S::kCols + c;
#pragma unroll
    for (int k = 0; k < kEpCols / 8; ++k) {
      uint32_t v[8];
      load32(q + 8 * k, v);
#pragma unroll
      for (int x = 0; x < 8; ++x) z[8 * k + x] += __uint_as_float(v[x]);
    }
  }
  if (a.ep.type == OB_TYPE_BF16)
    epilogue<__nv_bfloat16>(a.ep, z, m0, n0, a.M, a.N, turn[w]);
  else
    epilogue<__half>(a.ep, z, m0, n0, a.M, a.N, turn[w]);
}

constexpr int kSms = 152;

struct Plan {
  int cg, tiles_m, tiles_n, steps, workers, whole;
};

// What a product is cut into.  By sizes alone: the workspace goes by it.
Plan plan_of(int64_t M, int64_t N, int64_t K) {
  Plan p{};
  const int64_t steps = (K + BK - 1) / BK;
  const int64_t tm2 = (M + 255) / 256, tn2 = (N + 255) / 256;
  p.cg = tm2 * tn2 >= kSms / 4 ? 2 : 1;
  const int edge = 128 * p.cg;
  p.tiles_m = (int)((M + edge - 1) / edge);
  p.tiles_n = (int)((N + edge - 1) / edge);
  p.steps = (int)steps;
  const int most = kSms / p.cg;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  p.workers = (int)(tiles < most ? tiles : most);
  p.whole = steps ? (int)tiles : 0;
  if (!steps) return p;
  // Cutting the last tiles saves steps, and costs the second kernel and its traffic.
  const int64_t rest = tiles % most;
  if (rest) {
    const int64_t saved = p.steps - (rest * p.steps + most - 1) / most;
    if (saved > 16) {
      p.whole = (int)(tiles - rest);
      p.workers = most;
    }
  }
  return p;
}

template <int CG>
cudaError_t run(const Gemm& g, const Plan& p, cudaStream_t s) {
  using S = Shape<CG>;
  GemmArgs a{};
  cudaError_t e = cudaSuccess;
  if (p.steps) e = g.a_mn ? matrix_tensor_map(&a.a, g.a, g.ep.type, g.K, g.M, BK)
                         : matrix_tensor_map(&a.a, g.a, g.ep.type, g.M, g.K, 128);
  if (p.steps && e == cudaSuccess)
    e = g.b_mn ? matrix_tensor_map(&a.b, g.b, g.ep.type, g.K, g.N, BK)
               : matrix_tensor_map(&a.b, g.b, g.ep.type, g.N, g.K, 128);
  if (e != cudaSuccess) return e;
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
  const int rest = p.tiles_m * p.tiles_n - p.whole;
  const dim3 parts(rest * ((S::kRows / 32) * (S::kCols / kEpCols) / 8));
  if (!p.steps) return launch_behind(k_gemm_parts<CG>, parts, dim3(256), 0, s, a);
  static PerDeviceOnce once;
  e = once.run([] {
    return cudaFuncSetAttribute(k_gemm<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)S::kBytes);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(p.workers * CG);
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
  e = cudaLaunchKernelEx(&c, k_gemm<CG>, a);
  if (e != cudaSuccess || rest == 0) return e;
  return launch_behind(k_gemm_parts<CG>, parts, dim3(256), 0, s, a);
}

}  // namespace

size_t gemm_partial_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const Plan p = plan_of(M, N, K);
  if (p.whole == p.tiles_m * p.tiles_n || !p.steps) return 0;
  return (size_t)p.workers * 2 * (128 * p.cg) * (128 * p.cg) * sizeof(float);
}

cudaError_t launch_gemm(const Gemm& g, cudaStream_t s) {
  if (g.M == 0 || g.N == 0) return cudaSuccess;
  const Plan p = plan_of(g.M, g.N, g.K);
  return p.cg == 2 ? run<2>(g, p, s) : run<1>(g, p, s);
}

cudaError_t layer_error_word(unsigned** word) {
  static std::atomic<unsigned*> known[64];  // by device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  *word = known[dev & 63].load(std::memory_order_acquire);
  if (*word) return cudaSuccess;
  e = cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_layer_error);
  if (e == cudaSuccess) known[dev & 63].store(*word, std::memory_order_release);
  return e;
}

}  // namespace ob
