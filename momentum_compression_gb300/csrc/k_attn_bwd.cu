// Attention, backward.
//
//   P = exp(S scale + bias - lse), Z = P kept (0 or P), dP = do V^T
//   delta = rowsum(do o) / keep scale,  dS = Z dP - P delta
//   dv = keep scale Z^T do,  dq = scale keep scale dS K,  dk = ... dS^T Q
//   dtable[n][h] = keep scale * the sum of dS over the pairs of bucket n
//
// Three kernels, a fourth for few keys and a fifth for shared heads.  k_rows: -lse
// and -delta of every query.  k_attn_grad twice: for 128 queries at a time over
// the keys (dq and the bias table's sums), and for 128 keys at a time over the
// queries of the heads that share them (dk, dv).  Both recompute S and dP on the tensor
// cores and need no atomics: seven products instead of the five of a single
// pass, for results that are the same bits on every run.  k_join adds up heads
// that share keys where they were worked out one by one.
//
// A block holds its 128 rows X, Y in shared memory (q, do or k, v) and walks
// over tiles of 64 of the other side, U, W:
//   S = X U^T, dP = Y W^T   128 x 64 each in tensor memory
//   Z, dS                   from them in registers, rounded over S and dP
//   acc1 += Z W (dv), acc2 += dS U (dq or dk)    first operand from tensor memory
// Z and dS are rounded to the inputs' type, as the matrix unit wants them; all
// that is summed, and the bias table's sums, are fp32.
//
// delta is of the o that was stored: rounded, and the sum of rounded weights.
// Over many keys o is small, and its error in dq and dk well below that of dS's
// rounding.  Over few it is as large or larger (dq at 27 keys 1.95 times as far
// from 64 bits as with fp32 throughout, the bias table's gradient 2.4 times; two
// roundings are 1.42): there k_attn_grad runs a third time before the others
// (EXACT), for delta = sum of Z dP / sum of P, and drops the scores.
//
// Two tiles are in work at
// a time, each by two warpgroups (a thread a row of 32 columns), so one's
// arithmetic runs beside the other's products: sixteen warps that work, since a
// single one's dependent instructions leave three of four issue slots empty.
//
// A block stays on its SM and takes one piece of work (128 rows of X) after
// another from a counter, the products of the next begun before the last of
// this one are in.  Which block takes what changes no result.  Beside the
// warpgroups it has a warp each that issues the products of S and dP, those
// of the accumulators, and the copies (and clears the rows of pieces without
// pairs), and one that stages the bias of the next head and adds up the bias
// table's sums of the last.
//
// dq and the pass for dk and dv need nothing of one another (but the bias
// table's sums): the second's blocks start as the first's end (12 heads x 128
// queries x 128 keys 24.6 -> 16.2 us, 32 x 12 x 512 of d 64 309 -> 294 us).
//
// What bounds it is the issue of the arithmetic, not the matrix unit: without
// bias and dropout 897 TFLOP/s (five products counted) at d 128 x 8192 in
// 3.1 ms, 668 at d 64 x 2048 in 0.51 ms; with both, at 32 x 12 x 512 of
// d 64, 0.26 ms full (the two passes' keep bits alone are 48 us of every
// scheduler) and 0.24 ms over ragged lengths, where the start and the end of
// the many short pieces weigh more.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kRows = 128;  // rows of X, Y
constexpr int kTileRows = 64;
constexpr int kRowThreads = 256;   // of k_rows

struct GradArgs {
  CUtensorMap q, grad_o, k, v;  // boxes of 64 rows
  int B, H, Hkv, D, Lq, Lk, causal, q_offset, biased;
  int blocks, items;  // 128-row blocks of a head; blocks * batch * heads
  int sum_bufs;       // buffers of the bias table's sums, 0: none are wanted
  int exact_tiles;    // EXACT: the most tiles of a piece
  float scale, scale2;  // scale2 = scale * log2(e)
  ob_relpos rp;
  const void* table;
  const int32_t* kv_len;
  Keep keep;
  float* rows;     // of each tile of 64 queries: 64 times -lse * log2(e) (-inf: no weight),
                   // then 64 times -rowsum(do o) / keep.scale
  int Lqp;
  Heads out1, out2;  // dq: out2 = dq; dkv: out1 = dv, out2 = dk
  float* partial;    // [H][sum_parts][num_buckets]: dq writes them, dkv adds them into dtable
  int sum_parts;     // B * the blocks of dq
  void* dtable;      // dkv: or null
  float* join;       // dkv, split over the heads that share keys: [dv, dk][B][H][Lk][D], or null
  unsigned* next;    // the counter of this launch, 0 at its start
  bool behind_dq;    // dkv: launched behind dq
  unsigned* err;
};

struct RowArgs {
  int B, H, D, Lq, Lqp;
  Heads o, grad_o;
  const float* lse;
  float inv_keep;
  float* rows;
  unsigned* next;  // two counters to clear
};

// ---------------------------------------------------------------------------
// -lse and -rowsum(do o): a block takes 128 queries of a head, LANES lanes a
// row, four rows' loads on their way at once (32 x 12 x 512 of d 64, 50 MB, in
// 11 us; with a row at a time 23).  Rows past Lq and rows without keys get
// -lse = -inf, which makes every weight exp2(s - lse) zero.
// ---------------------------------------------------------------------------

// Where query i of head bh has the first of its two values; the second is
// kTileRows further.
__device__ __forceinline__ int64_t row_at(int bh, int Lqp, int i) {
  return (int64_t)bh * Lqp * 2 + (int64_t)(i / kTileRows) * (2 * kTileRows) + i % kTileRows;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(kRowThreads) k_rows(const RowArgs a) {
  grid_release();
  if (blockIdx.x == 0 && threadIdx.x < 2) a.next[threadIdx.x] = 0;
  const int heads = a.B * a.H;
  if (heads == 0 || a.Lq == 0) return;
  constexpr int kPass = kRowThreads / LANES, N = 4;
  const int l = threadIdx.x % LANES, r0 = (int)(blockIdx.x / heads) * kRows + threadIdx.x / LANES;
  const int bh = blockIdx.x % heads, b = bh / a.H, h = bh % a.H;
  const T* o = static_cast<const T*>(a.o.data) + b * a.o.b + h * a.o.h + 8 * l;
  const T* g = static_cast<const T*>(a.grad_o.data) + b * a.grad_o.b + h * a.grad_o.h + 8 * l;
#pragma unroll 1
  for (int p = r0; p < r0 / kRows * kRows + kRows; p += N * kPass) {
    uint4 x[N], y[N];
    float lse[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = p + n * kPass;
      x[n] = y[n] = make_uint4(0, 0, 0, 0);
      lse[n] = -INFINITY;
      if (i >= a.Lq) continue;
      if (8 * l < a.D) {
        x[n] = *reinterpret_cast<const uint4*>(o + (int64_t)i * a.o.l);
        y[n] = *reinterpret_cast<const uint4*>(g + (int64_t)i * a.grad_o.l);
      }
      lse[n] = a.lse[(int64_t)bh * a.Lq + i];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t xs[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      const uint32_t ys[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<T>(xs[k]), e = unpack2<T>(ys[k]);
        sum = __fmaf_rn(f.x, e.x, sum);
        sum = __fmaf_rn(f.y, e.y, sum);
      }
#pragma unroll
      for (int k = LANES / 2; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if (l == 0) {
        const bool none = lse[n] == -INFINITY;
        float* to = a.rows + row_at(bh, a.Lqp, p + n * kPass);
        to[0] = none ? -INFINITY : -lse[n] * kLog2e;
        to[kTileRows] = none ? 0.0f : -sum * a.inv_keep;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The gradients
// ---------------------------------------------------------------------------

template <int DP, bool DQ>
struct GradShape {
  static constexpr int kGroups = 4;  // warpgroups, two a tile
  // Tiles whose S and dP are in tensor memory: with a third, the scores of a
  // pair's next tile are there when it is done with one (d 64 x 2048 backward
  // 702 -> 565 us).  At 128 there is no room for it, or for its stage.
  static constexpr int kSlots = DP == 64 ? 3 : 2;
  static constexpr int kStages = DP == 64 ? 5 : 3;
  static constexpr int kXBufs = DP == 64 ? 2 : 1;
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (kWarps + 4);  // and the four warps of the other roles
  static constexpr uint32_t kX = kRows * DP * 2;
  static constexpr uint32_t kTile = kTileRows * DP * 2;
  static constexpr uint32_t kStage = 2 * kTile + (DQ ? 0 : 1024);  // U, W and the queries' rows
  static constexpr uint32_t kRing = kXBufs * 2 * kX;               // offset of the stages
  static constexpr uint32_t kBias = kRing + kStages * kStage;      // of two biases, then the sums
  // tensor memory: S and dP of each slot, one or two sets of accumulators
  static constexpr uint32_t kAcc = 128 * kSlots, kAccCols = DQ ? DP : 2 * DP;
  static constexpr int kAccBufs = (512 - kAcc) / kAccCols >= 2 ? 2 : 1;
  static constexpr int kExactFloats = 2 * kGroups * kRows;  // EXACT: a buffer of its sums
  // floats of one buffer of sums: by distance for each warp, and of each
  // group's rows eps, far left and right, mass left and right
  __host__ __device__ static constexpr int sum_floats(int ndist) {
    return kWarps * ndist + 5 * kGroups * kRows;
  }
};

// Sums by distance cover this much past the outermost buckets' edges: all that
// a block of 32 x 16 touches when it touches what lies between them.
constexpr int kSumMargin = 48;

// Floats of a staged bias of n distances, and distances of the sums that go
// with it: in whole float4.
__host__ __device__ constexpr int bias_room(int n) { return (n + 3) / 4 * 4; }
__host__ __device__ constexpr int sum_dists(int n) {
  return (n - 2 * (kBiasMargin - kSumMargin) + 3) / 4 * 4;
}

constexpr int kItems = 4;  // pieces handed out at a time

// Tiles of keys up to which a piece's delta is worked out from the scores.  Of 60
// drawn training calls 37 were over 1.5 times as far from 64 bits as with fp32
// throughout when none was, of 450 ten with these, by up to 1.56.  The bias table's
// gradient, which is not rounded on the way, wants more of them (256 keys: 1.9
// times with two, 1 with four) but where a batch is of longer and shorter entries.
// It costs the backward pass of 32 x 12 x 512, lengths from 128 on, 227 -> 239 us
// (four tiles 250), 32 x 12 x 256 with a table 99 -> 131 (without one nothing;
// four tiles 87 -> 116), 32 x 12 x 128 44 -> 55, 8 x 2048 causal of d 128 542 -> 551.
constexpr int kExactTiles = 2, kExactTilesTable = 4;

struct Item {
  int x0, b, hx, keys, from, per;  // x0 < 0: no more
};

template <int W, int S>
struct GradBars {
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t x_full[2], x_empty[2], full[S], empty[S], s_full[3], p_full[3], acc_full[2], acc_free[2];
  uint64_t bias_full[2], bias_empty[2], sums_full[2], sums_empty[2], drain[2];
  Item item[kItems], done[W];  // done: the piece whose results a warp still has to take
  alignas(16) float rows[kItems][2 * kRows];  // dq: of the piece's queries, as in global memory
  uint32_t tmem;
  int first[OB_RELPOS_MAX_SIDE];
  uint8_t bucket[kBiasMost];
  alignas(16) float carry[W][16];
};

// The pair of weights whose halfwords are w, dropped ones as zero.
__device__ __forceinline__ void keep_pair(uint32_t w, uint32_t T2, float p0, float p1, float* z0,
                                          float* z1) {
  asm("{\n\t.reg .pred a, b;\n\t.reg .b32 u;\n\t"
      "abs.bf16x2 u, %2;\n\t"
      "setp.geu.bf16x2 a|b, u, %3;\n\t"
      "selp.f32 %0, %4, 0f00000000, a;\n\t"
      "selp.f32 %1, %5, 0f00000000, b;\n\t}"
      : "=f"(*z0), "=f"(*z1)
      : "r"(w), "r"(T2), "f"(p0), "f"(p1));
}

// v += what the lane below (lane - 1) has in u; in lane 0 nothing.
__device__ __forceinline__ void add_from_below(float* v, float u) {
  asm volatile("{\n\t.reg .pred in;\n\t.reg .f32 t;\n\t"
               "shfl.sync.up.b32 t|in, %1, 1, 0, 0xffffffff;\n\t"
               "@in add.f32 %0, %0, t;\n\t}"
               : "+f"(*v)
               : "f"(u));
}

// Keep bits of 32 queries for the thread's key, from calls that hold eight
// keys of one query: lane l draws the queries 8 k + l % 8 (call0 of k = 0, a
// query further every `step` calls) for the eight keys of its eight lanes,
// and an 8 x 8 transposition of bits among those lanes turns query numbers
// into bit numbers.  Bit r: query r.
__device__ __forceinline__ uint32_t keep_column(const Keep& keep, uint64_t call0, uint32_t step,
                                                int lane) {
  uint32_t x = 0, y = 0;  // queries 8 k + l % 8 for k = 0, 1 and for k = 2, 3
  uint4 w[4];
  keep_words_n(keep, call0, 8 * step, w);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    uint32_t& to = k < 2 ? x : y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      to |= keep_mask2(u[e], keep.T * 0x10001u) & (0x00020001u << (2 * e + 8 * (k & 1)));
  }
  // even keys are in the low halves, odd ones in the high halves
  uint32_t v = __byte_perm(x, y, 0x5410) | __byte_perm(x, y, 0x7632);
#pragma unroll
  for (int s = 4; s; s >>= 1) {
    const uint32_t low = s == 4 ? 0x0f0f0f0fu : s == 2 ? 0x33333333u : 0x55555555u;
    const bool up = lane & s;
    const uint32_t o = __shfl_xor_sync(0xffffffffu, v, s);
    v = up ? (v & ~low) | (o >> s & low) : (v & low) | (o << s & ~low);
  }
  return v;
}

// EXACT (with DQ): delta alone, for pieces of at most exact_tiles tiles of keys.
template <typename T, int DP, bool DQ, bool DROP, bool EXACT>
__global__ void __launch_bounds__(GradShape<DP, DQ>::kThreads, 1)
    k_attn_grad(const __grid_constant__ GradArgs a) {
  static_assert(DQ || !EXACT, "");
  using S = GradShape<DP, DQ>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int G = S::kGroups, K = S::kSlots;
  constexpr int kScores = 4 * G, kProducts = kScores + 1, kCopies = kScores + 2;
  extern __shared__ uint8_t raw[];
  __shared__ GradBars<S::kWarps, S::kStages> bar;
  uint8_t* smem = align_shared(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const BiasSpan span = a.biased ? bias_span(a.rp) : BiasSpan{0, 0};
  const int nbias = a.biased ? bias_floats(a.rp) : 0;
  const int bias_step = DQ ? bias_room(nbias) : nbias;  // the sums behind them are read as float4
  const int ndist = a.biased ? sum_dists(nbias) : 0;
  // A piece's heads: its X, the first and the number of those on the other side.
  const int group = a.H / a.Hkv;
  const bool single = DQ || a.join;
  const int heads_x = single ? a.H : a.Hkv, heads = single ? 1 : group;
  float* biases = reinterpret_cast<float*>(smem + S::kBias);
  float* sums = biases + 2 * bias_step;  // sum_bufs buffers of sum_size
  const int sum_size = EXACT ? S::kExactFloats : S::sum_floats(ndist);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], (EXACT ? 2 : 2 + (a.biased ? 1 : 0)) + S::kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.x_full[i], 1);
      mbar_init(&bar.x_empty[i], 1);
      mbar_init(&bar.bias_full[i], 1);
      mbar_init(&bar.bias_empty[i], S::kWarps);
      mbar_init(&bar.sums_full[i], S::kWarps);
      mbar_init(&bar.sums_empty[i], 1);
      mbar_init(&bar.drain[i], 1);
      mbar_init(&bar.acc_full[i], 1);
      mbar_init(&bar.acc_free[i], S::kWarps);
    }
    for (int i = 0; i < K; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], S::kWarps / 2);
    }
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], EXACT ? S::kWarps / 2 : 1);
    }
    fence_barrier_init();
  }
  if (warp == kProducts) tmem_alloc(&bar.tmem, 512);
  if (a.biased) {
    for (int i = threadIdx.x; i < a.rp.side; i += S::kThreads) bar.first[i] = a.rp.first[i];
    stage_buckets(bar.bucket, a.rp, threadIdx.x, S::kThreads);
    for (int i = threadIdx.x; i < a.sum_bufs * sum_size; i += S::kThreads) sums[i] = 0.0f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  // dk and dv need nothing of dq's before the bias table's sums: they start as
  // its blocks end, which have all waited for the rows.
  if (DQ || !a.behind_dq) grid_wait();
  grid_release();

  // The k-th piece of work of this block, for one of the roles that follow it:
  // false after the last, or when the wait ran out.
  auto take = [&](int k, Item& it, auto&& use) {
    const int slot = k % kItems;
    if (!warp_wait(&bar.item_full[slot], (k / kItems) & 1, a.err)) return false;
    it = bar.item[slot];
    use(slot);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.item_empty[slot]);
    return it.x0 >= 0;
  };

  if (warp == kCopies) {
    // ----- copies --------------------------------------------------------
    // DQ: x0 is a query of head hx.  Else a key of head hx, and the tiles run over
    // the queries from tile `from` on of the heads that share it.
    int idx = blockIdx.x, k = 0, nx = 0, nt = 0;  // pieces, X buffers and tiles issued so far
    int given = 0;                                // of the pieces, those that were handed out
    bool ok = true;
    // Finds the next piece with pairs, clearing the rows of those without, and
    // hands it to the other roles.
    auto hand_out = [&] {
      Item it{-1, 0, 0, 0, 0, 0};
      while (idx < a.items) {
        // Causal: the last queries see the most keys, the first keys the most queries.
        const int blk = idx / (a.B * heads_x), bh = idx % (a.B * heads_x);
        const int x0 = (DQ && !EXACT ? a.blocks - 1 - blk : blk) * kRows, b = bh / heads_x,
                  hx = bh % heads_x;
        unsigned n = 0;
        if (EXACT)  // pieces much alike, most of which may be passed over: in turn
          n = idx + gridDim.x;
        else if (lane == 0)
          n = gridDim.x + atomicAdd(a.next, 1u);
        const int keys = key_count(a, b);
        int from = 0, per;
        if (DQ) {
          int last = keys;
          if (a.causal) last = min(last, min(x0 + kRows, a.Lq) + a.q_offset);
          per = last > 0 ? (last + kTileRows - 1) / kTileRows : 0;
        } else {
          if (a.causal) from = max(0, x0 - a.q_offset) / kTileRows;
          per = x0 < keys ? max(0, (a.Lq + kTileRows - 1) / kTileRows - from) : 0;
        }
        idx = (int)__shfl_sync(0xffffffffu, n, 0);
        if (per > 0 && (!EXACT || per <= a.exact_tiles)) {
          it = Item{x0, b, hx, keys, from, per};
          break;
        }
        if (EXACT) continue;
        // 16 bytes a lane, as many rows at a time as a warp has lanes for.
        const int chunks = a.D / 8, each = 32 / chunks, d = lane % chunks * 8;
        const int rows = lane < each * chunks ? min(kRows, (DQ ? a.Lq : a.Lk) - x0) : 0;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        if (!DQ && a.join) {
          float* dv = a.join + (((int64_t)b * a.H + hx) * a.Lk + x0) * a.D + d;
          float* dk = dv + (int64_t)a.B * a.H * a.Lk * a.D;
          for (int r = lane / chunks; r < rows; r += each)
            for (int half = 0; half < 8; half += 4) {
              *reinterpret_cast<uint4*>(dv + r * a.D + half) = zero;
              *reinterpret_cast<uint4*>(dk + r * a.D + half) = zero;
            }
        } else {
          T* to2 = static_cast<T*>(a.out2.data) + b * a.out2.b + x0 * a.out2.l + hx * a.out2.h + d;
          T* to1 = static_cast<T*>(a.out1.data) + b * a.out1.b + x0 * a.out1.l + hx * a.out1.h + d;
#pragma unroll 4
          for (int r = lane / chunks; r < rows; r += each) {
            *reinterpret_cast<uint4*>(to2 + r * a.out2.l) = zero;
            if (!DQ) *reinterpret_cast<uint4*>(to1 + r * a.out1.l) = zero;
          }
        }
        if (DQ && a.sum_bufs) {
          float* to =
              a.partial + (((int64_t)hx * a.B + b) * a.blocks + x0 / kRows) * a.rp.num_buckets;
          for (int i = lane; i < a.rp.num_buckets; i += 32) to[i] = 0.0f;
        }
      }
      const int slot = k % kItems;
      if (k >= kItems)
        ok = warp_wait(&bar.item_empty[slot], (k / kItems + 1) & 1, a.err, kErrWaitEmpty);
      if (ok) given = k + 1;
      if (ok && lane == 0) {
        bar.item[slot] = it;
        if (DQ && it.x0 >= 0) {
          constexpr uint32_t bytes = 2 * kRows * sizeof(float);  // Lqp covers every row
          mbar_arrive_expect_tx(&bar.item_full[slot], bytes);
          bulk_g2s(bar.rows[slot], a.rows + row_at(it.b * a.H + it.hx, a.Lqp, it.x0), bytes,
                   &bar.item_full[slot]);
        } else {
          mbar_arrive(&bar.item_full[slot]);
        }
      }
      ++k;
      return it;
    };
    Item it = hand_out(), after{-1, 0, 0, 0, 0, 0};
    while (ok && it.x0 >= 0) {
      const int xb = nx % S::kXBufs;
      if (nx >= S::kXBufs)
        ok = warp_wait(&bar.x_empty[xb], (nx / S::kXBufs + 1) & 1, a.err, kErrWaitEmpty);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bar.x_full[xb], 2 * S::kX);
        const int h = !DQ && a.join ? it.hx / group : it.hx;
        for (int x = 0; x < DP / 64; ++x)
          for (int r = 0; r < kRows; r += kTileRows) {
            uint8_t* to = smem + xb * 2 * S::kX + x * (kRows * 128) + r * 128;
            tma_load4(to, DQ ? &a.q : &a.k, 64 * x, it.x0 + r, h, it.b, &bar.x_full[xb]);
            tma_load4(to + S::kX, DQ ? &a.grad_o : &a.v, 64 * x, it.x0 + r, h, it.b,
                      &bar.x_full[xb]);
          }
      }
      ++nx;
      for (int hh = 0; ok && hh < heads; ++hh) {
        const int hu = DQ ? it.hx / group : a.join ? it.hx : it.hx * group + hh;
        for (int t = 0; t < it.per; ++t, ++nt) {
          const int st = nt % S::kStages;
          if (nt >= S::kStages)
            ok = warp_wait(&bar.empty[st], (nt / S::kStages + 1) & 1, a.err, kErrWaitEmpty);
          if (!ok) break;
          uint8_t* to = smem + S::kRing + st * S::kStage;
          const int r = (it.from + t) * kTileRows;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bar.full[st], 2 * S::kTile + (DQ ? 0 : kTileRows * 8));
            for (int x = 0; x < DP / 64; ++x) {
              tma_load4(to + x * (kTileRows * 128), DQ ? &a.k : &a.q, 64 * x, r, hu, it.b,
                        &bar.full[st]);
              tma_load4(to + S::kTile + x * (kTileRows * 128), DQ ? &a.v : &a.grad_o, 64 * x, r,
                        hu, it.b, &bar.full[st]);
            }
            if (!DQ)
              bulk_g2s(to + 2 * S::kTile, a.rows + row_at(it.b * a.H + hu, a.Lqp, r),
                       kTileRows * 8, &bar.full[st]);
          }
          // The next piece is found while the first tiles are on their way.
          if (hh == 0 && t == min(it.per, 2) - 1) after = hand_out();
          if (!ok) {
            ++nt;
            break;
          }
        }
      }
      it = after;
    }
    // Whatever became of the others: what is in flight lands before the block ends.
    for (int i = max(0, nx - S::kXBufs); i < nx; ++i)
      mbar_wait(&bar.x_full[i % S::kXBufs], (i / S::kXBufs) & 1, a.err, kErrDrain);
    for (int i = max(0, nt - S::kStages); i < nt; ++i)
      mbar_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1, a.err, kErrDrain);
    for (int i = max(0, given - kItems); i < given; ++i)
      mbar_wait(&bar.item_full[i % kItems], (i / kItems) & 1, a.err, kErrDrain);
  } else if (warp == kScores) {
    // ----- S and dP -------------------------------------------------------
    constexpr uint32_t kShapeS = mma_shape(kBf16, kTileRows, false);
    const uint32_t leader = elect_lane();
    const uint64_t x_desc = desc_k(smem_u32(smem)), u_desc = desc_k(smem_u32(smem) + S::kRing);
    const int ksteps = (a.D + 15) / 16;
    bool ok = true;
    int st = 0, par = 0, g = 0;     // stage, its phase, slot of the tile
    int fst = 0, fpar = 0, nt = 0;  // stage and phase of the tile that had the slot last
    Item it;
    for (int k = 0; ok && take(k, it, [](int) {}); ++k) {
      const int xb = k % S::kXBufs;
      ok = warp_wait(&bar.x_full[xb], (k / S::kXBufs) & 1, a.err);
      const uint64_t xd = x_desc + (uint32_t)xb * (2 * S::kX >> 4);
      const int total = heads * it.per;
      for (int t = 0; ok && t < total; ++t, ++nt) {
        ok = warp_wait(&bar.full[st], par, a.err);
        // Once that tile's products are done, its P and dS may be written over.
        if (ok && nt >= K) {
          ok = warp_wait(&bar.empty[fst], fpar, a.err, kErrWaitEmpty);
          if (++fst == S::kStages) fst = 0, fpar ^= 1;
        }
        if (!ok) break;
        tc_fence_after();
        const uint64_t ud = u_desc + (uint32_t)st * (S::kStage >> 4);
        const uint32_t d = tmem + g * 128;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int s = 0; s < DP / 16; ++s)
            if (s < ksteps)
              mma_ss(leader, d + 64 * y,
                     xd + ((y * S::kX + (s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4),
                     ud + ((y * S::kTile + (s >> 2) * (kTileRows * 128) + (s & 3) * 32) >> 4),
                     kShapeS, s > 0);
        mma_commit(leader, &bar.s_full[g]);
        if (++st == S::kStages) st = 0, par ^= 1;
        if (++g == K) g = 0;
      }
      mma_commit(leader, &bar.x_empty[xb]);
    }
    // Nothing may arrive after the block's end.
    mma_commit(leader, &bar.drain[0]);
    mbar_wait(&bar.drain[0], 0, a.err, kErrDrain);
  } else if (warp == kProducts && !EXACT) {
    // ----- the accumulators -----------------------------------------------------
    constexpr uint32_t kShapeA = mma_shape(kBf16, DP, true);
    const uint32_t leader = elect_lane();
    const uint64_t u_rows = desc_mn(smem_u32(smem) + S::kRing, kTileRows * 128);
    bool ok = true;
    int st = 0, g = 0, gpar = 0;
    Item it;
    for (int k = 0; ok && take(k, it, [](int) {}); ++k) {
      const int total = heads * it.per, ab = k % S::kAccBufs;
      const uint32_t acc = tmem + S::kAcc + ab * S::kAccCols;
      for (int t = 0; t < total; ++t) {
        ok = warp_wait(&bar.p_full[g], gpar, a.err);
        if (ok && t == 0 && k >= S::kAccBufs)
          ok = warp_wait(&bar.acc_free[ab], (k / S::kAccBufs + 1) & 1, a.err, kErrWaitEmpty);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ud = u_rows + (uint32_t)st * (S::kStage >> 4);
        const uint32_t p = tmem + g * 128;
        // The tile's warpgroups each left 32 rows of the sum over their own columns.
        if (!DQ) {
#pragma unroll
          for (int s = 0; s < kTileRows / 16; ++s)
            mma_ts(leader, acc, p + (s >> 1) * 32 + (s & 1) * 8,
                   ud + ((S::kTile + s * 2048) >> 4), kShapeA, t > 0 || s > 0);
        }
#pragma unroll
        for (int s = 0; s < kTileRows / 16; ++s)
          mma_ts(leader, acc + (DQ ? 0 : DP), p + 64 + (s >> 1) * 32 + (s & 1) * 8,
                 ud + (s * 2048 >> 4), kShapeA, t > 0 || s > 0);
        mma_commit(leader, &bar.empty[st]);
        if (++st == S::kStages) st = 0;
        if (++g == K) g = 0, gpar ^= 1;
      }
      if (ok) mma_commit(leader, &bar.acc_full[ab]);
    }
    mma_commit(leader, &bar.drain[1]);
    mbar_wait(&bar.drain[1], 0, a.err, kErrDrain);
  } else if (warp > kCopies) {
    // ----- helper: the biases ahead, the bias table's sums behind -----------------
    if (EXACT || a.biased) {
      int k = 0, nb = 0;  // pieces taken, biases staged
      bool ok = true;
      Item it, prev;
      bool have = take(k, it, [](int) {}), had = false;
      int done = 0;  // pieces whose sums are out
      // The distances of bucket n, and those of the lane's first.
      auto distances = [&](int n) {
        int64_t lo, hi;
        bucket_range(bar.first, a.rp.side, a.rp.two_sided, n, -(span.left + kSumMargin),
                     span.right + kSumMargin, &lo, &hi);
        return make_int2((int)lo, (int)hi);
      };
      int2 mine = make_int2(0, 0);
      if (DQ && !EXACT && a.sum_bufs && lane < a.rp.num_buckets) mine = distances(lane);
      while (ok && (have || had)) {
        if (have) {
          ++k;
          for (int hh = 0; ok && a.biased && hh < heads; ++hh, ++nb) {
            if (nb >= 2)
              ok = warp_wait(&bar.bias_empty[nb & 1], (nb / 2 + 1) & 1, a.err, kErrWaitEmpty);
            if (!ok) break;
            stage_bias(biases + (nb & 1) * bias_step, bar.bucket, nbias,
                       static_cast<const T*>(a.table), a.H, single ? it.hx : it.hx * group + hh,
                       lane, 32);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.bias_full[nb & 1]);
          }
        }
        if (EXACT && had && ok) {
          const int sb = done % a.sum_bufs;
          ok = warp_wait(&bar.sums_full[sb], (done / a.sum_bufs) & 1, a.err);
          if (!ok) break;
          const float* row = sums + sb * sum_size;  // [sum of P, of Z dP][G][kRows]
          for (int r = lane; r < kRows; r += 32) {
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int g = 0; g < G; ++g) v[i] += row[(i * G + g) * kRows + r];
            // Rows of no weight (past Lq, without keys) keep the 0 of k_rows.
            if (v[0] != 0.0f)
              a.rows[row_at(prev.b * a.H + prev.hx, a.Lqp, prev.x0 + r) + kTileRows] = -v[1] / v[0];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sums_empty[sb]);
          ++done;
        }
        if (!EXACT && had && ok && DQ && a.sum_bufs) {
          const int sb = done % a.sum_bufs;
          ok = warp_wait(&bar.sums_full[sb], (done / a.sum_bufs) & 1, a.err);
          if (!ok) break;
          float* by_d = sums + sb * sum_size;
          float* row = by_d + S::kWarps * ndist;  // [5][G][kRows]
          // A row's dS sums to zero; what it sums to is the error of rowsum(do o),
          // where that is of the rounded o.  It is taken out of the far buckets, whose
          // weight would multiply it.
          float far_l = 0.0f, far_r = 0.0f;
          for (int r = lane; r < kRows; r += 32) {
            float v[5] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 5; ++i)
#pragma unroll
              for (int g = 0; g < G; ++g) v[i] += row[(i * G + g) * kRows + r];
            far_l += v[1] - v[0] * v[3];
            far_r += v[2] - v[0] * v[4];
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            far_l += __shfl_xor_sync(0xffffffffu, far_l, o);
            far_r += __shfl_xor_sync(0xffffffffu, far_r, o);
          }
          // The warps' sums of a distance into the first warp's, the others cleared.
          for (int i = lane; i < ndist / 4; i += 32) {
            float4* d = reinterpret_cast<float4*>(by_d) + i;
            float4 sum[2] = {d[0], d[ndist / 4]};
#pragma unroll
            for (int w = 2; w < S::kWarps; ++w) {
              const float4 v = d[w * (ndist / 4)];
              float4& to = sum[w & 1];
              to = make_float4(to.x + v.x, to.y + v.y, to.z + v.z, to.w + v.w);
            }
#pragma unroll
            for (int w = 1; w < S::kWarps; ++w)
              d[w * (ndist / 4)] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            d[0] = make_float4(sum[0].x + sum[1].x, sum[0].y + sum[1].y, sum[0].z + sum[1].z,
                               sum[0].w + sum[1].w);
          }
          __syncwarp();
          float* to = a.partial + (((int64_t)prev.hx * a.B + prev.b) * a.blocks + prev.x0 / kRows) *
                                      a.rp.num_buckets;
          for (int n = lane; n < a.rp.num_buckets; n += 32) {
            const int2 of = n == lane ? mine : distances(n);
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (n == a.rp.side - 1) sum[0] = far_l;
            if (n == (a.rp.two_sided ? a.rp.num_buckets - 1 : 0)) sum[1] = far_r;
            const float* from = by_d + span.left + kSumMargin;
            int i = of.x;
            for (; i + 4 <= of.y; i += 4)
#pragma unroll
              for (int j = 0; j < 4; ++j) sum[j] += from[i + j];
            for (; i < of.y; ++i) sum[2] += from[i];
            to[n] = ((sum[0] + sum[1]) + (sum[2] + sum[3])) * a.keep.scale;
          }
          __syncwarp();
          for (int i = lane; i < ndist; i += 32) by_d[i] = 0.0f;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sums_empty[sb]);
          ++done;
        }
        had = have;
        prev = it;
        have = have && take(k, it, [](int) {});
      }
      // The bias table's gradient from the sums that dq left: a lane a bucket, in
      // order, beside the last piece's arithmetic.
      if (!DQ) grid_wait();
      if (!DQ && a.dtable)
        for (int h = blockIdx.x; h < a.H; h += gridDim.x)
          for (int n = lane; n < a.rp.num_buckets; n += 32) {
            const float* from = a.partial + (int64_t)h * a.sum_parts * a.rp.num_buckets + n;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int i = 0; i < a.sum_parts; ++i) sum[i & 3] += from[(int64_t)i * a.rp.num_buckets];
            static_cast<T*>(a.dtable)[(size_t)n * a.H + h] =
                from_f32<T>((sum[0] + sum[1]) + (sum[2] + sum[3]));
          }
    }
  } else if (!EXACT || warp < kScores) {
    // ----- arithmetic: a thread a row of X ----------------------------------
    const int g = warp >> 2, half = g & 1, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t per_row = (uint32_t)((a.Lk + 7) / 8);
    const uint32_t T2 = a.keep.T * 0x10001u;
    bool ok = true;
    // tiles of earlier pieces, the pair's next tile, biases used
    int nt = 0, next = g >> 1, nb = 0;
    float nlse = 0.0f, ndelta = 0.0f;  // of the row's query
    auto fetch = [&](int slot) {
      if (!DQ) return;
      const float* r = bar.rows[slot] + row_at(0, 0, row);
      nlse = r[0];
      ndelta = r[kTileRows];
    };
    // The results of piece kp, 16 columns at a time, the groups in turn.
    auto finish = [&](int kp) {
      const int ab = kp % S::kAccBufs;
      ok = warp_wait(&bar.acc_full[ab], (kp / S::kAccBufs) & 1, a.err);
      if (!ok) return;
      tc_fence_after();
      const Item done = bar.done[warp];
      const int x = done.x0 + row;
      const bool none = !DQ && x >= done.keys;
      constexpr int kMine = S::kAccCols / 16 / G;
      const uint32_t acc = tmem + lanes + S::kAcc + ab * S::kAccCols;
      // Of chunk c: whether it is of the second output, and its first column.
      auto second = [](int c) { return DQ || c >= DP / 16; };
      auto column = [](int c) { return 16 * (DQ ? c : c % (DP / 16)); };
      if (!DQ && a.join) {
#pragma unroll 1
        for (int i = 0; i < kMine; ++i) {
          const int c = g + i * G;
          uint32_t r[16];
          tmem_ld16(r, acc + 16 * c);
          tmem_wait_ld(r);
          const float mul = none ? 0.0f : second(c) ? a.scale * a.keep.scale : a.keep.scale;
          float* to = a.join +
                      (((int64_t)(second(c) * a.B + done.b) * a.H + done.hx) * a.Lk + x) * a.D +
                      column(c);
#pragma unroll
          for (int n = 0; n < 16; n += 4)
            if (x < a.Lk && column(c) + n < a.D)
              *reinterpret_cast<float4*>(to + n) =
                  none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                       : make_float4(__uint_as_float(r[n]) * mul, __uint_as_float(r[n + 1]) * mul,
                                     __uint_as_float(r[n + 2]) * mul,
                                     __uint_as_float(r[n + 3]) * mul);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.acc_free[ab]);
        return;
      }
      uint32_t o[kMine][8];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int c = g + i * G;
        uint32_t r[16];
        tmem_ld16(r, acc + 16 * c);
        tmem_wait_ld(r);
        const float mul = second(c) ? a.scale * a.keep.scale : a.keep.scale;
#pragma unroll
        for (int n = 0; n < 8; ++n)
          o[i][n] = none ? 0u
                         : pack2<T>(__uint_as_float(r[2 * n]) * mul,
                                    __uint_as_float(r[2 * n + 1]) * mul);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.acc_free[ab]);
      if (x < (DQ ? a.Lq : a.Lk)) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int c = g + i * G, col = column(c);
          const Heads& out = second(c) ? a.out2 : a.out1;
          T* to = static_cast<T*>(out.data) + done.b * out.b + (int64_t)x * out.l +
                  done.hx * out.h + col;
          if (col < a.D)
            *reinterpret_cast<uint4*>(to) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
          if (col + 8 < a.D)
            *reinterpret_cast<uint4*>(to + 8) = make_uint4(o[i][4], o[i][5], o[i][6], o[i][7]);
        }
      }
    };
    // A piece's results are taken after the first tile of the next: until then the
    // other groups' last tiles and their products would be waited for.
    Item it;
    bool have = take(0, it, fetch), pending = false;
    for (int k = 0; ok && (have || pending); ++k) {
      if (have) {
        const int x = it.x0 + row, wx = it.x0 + (warp & 3) * 32;  // the warp's first row
        const int h0 = single ? it.hx : it.hx * group, keys = it.keys;
        // The live columns of the row: DQ: below `limit`; else from `limit` on.
        int limit, warp_limit;
        if (DQ) {
          limit = a.causal ? min(keys, x + a.q_offset + 1) : keys;
          warp_limit = a.causal ? min(keys, wx + a.q_offset + 1) : keys;
        } else {
          limit = x >= keys ? INT32_MAX : a.causal ? x - a.q_offset : INT32_MIN;
          warp_limit = wx + 31 >= keys ? INT32_MAX : a.causal ? wx + 31 - a.q_offset : INT32_MIN;
        }
        float eps = 0.0f, far_l = 0.0f, far_r = 0.0f, mass_l = 0.0f, mass_r = 0.0f;
        float* by_d = sums;
        if (DQ && a.sum_bufs) {
          const int sb = k % a.sum_bufs;
          if (k >= a.sum_bufs)
            ok = warp_wait(&bar.sums_empty[sb], (k / a.sum_bufs + 1) & 1, a.err, kErrWaitEmpty);
          if (!ok) break;
          by_d = sums + sb * sum_size;
        }
        for (int hh = 0; ok && hh < heads; ++hh) {
          const float* bias = biases + (nb & 1) * bias_step;
          float far_left = 0.0f, far_right = 0.0f;
          if (a.biased) {
            ok = warp_wait(&bar.bias_full[nb & 1], (nb / 2) & 1, a.err);
            if (!ok) break;
            far_left = bias[0];
            far_right = bias[nbias - 1];
          }
          // Keep bits: the call of the row's first key, or of its key and query lane % 8.
          const uint64_t call0 =
              DQ ? ((uint64_t)(it.b * a.H + h0 + hh) * a.Lq + x) * per_row
                 : ((uint64_t)(it.b * a.H + h0 + hh) * a.Lq + (lane & 7)) * per_row + (x >> 3);
          for (; ok && next < nt + (hh + 1) * it.per; next += 2) {
            const int st = next % S::kStages, slot = next % K;
            const uint32_t ts = tmem + lanes + slot * 128 + half * 32, tp = ts + 64;
            // first of the group's 32 columns (keys or queries)
            const int c0 = (it.from + next - nt - hh * it.per) * kTileRows + 32 * half;
            uint8_t* stage = smem + S::kRing + st * S::kStage;
            uint32_t kept = ~0u;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {  // 16 columns at a time
              const int col = c0 + 16 * c;
              // The keep bits do not wait for the scores.
              uint4 words[2];
              if (DQ && DROP)
                keep_words_n(a.keep, call0 + (uint32_t)(col >> 3), 1, words);
              if (c == 0) {
                if (!DQ && DROP)
                  kept = keep_column(a.keep, call0 + (uint64_t)(uint32_t)c0 * per_row, per_row,
                                     lane);
                ok = warp_wait(&bar.s_full[slot], (next / K) & 1, a.err);
                if (!ok) break;
                tc_fence_after();
              }
              uint32_t vs[16], vp[16];
              tmem_ld16(vs, ts + 16 * c);
              tmem_ld16(vp, tp + 16 * c);
              // Distances of the warp's rows and the columns: [low, low + 46].
              const int low = (DQ ? col - wx - 31 : wx - col - 15) - a.q_offset;
              const bool near = a.biased && low + 46 > -span.left && low < span.right;
              const float far = !a.biased ? 0.0f : low >= span.right ? far_right : far_left;
              const bool masked = DQ ? col + 16 > warp_limit : col < warp_limit;

              // Z and dS of the columns.  Branch-free inside, for the scheduler's sake: a
              // body each for blocks of one bias value, blocks across several, and
              // blocks with masked pairs (of either kind).  No more is unrolled than
              // this: the warps of a block are all at different places of the code,
              // and more of it than the instruction caches hold costs more than it
              // saves.
              auto weigh = [&](auto several_t, auto mask_t) {
                constexpr bool kSeveral = decltype(several_t)::value;
                constexpr bool kMask = decltype(mask_t)::value;
                // The bias of column n of the row: tb[n * step].
                const int step = (kSeveral || near) ? (DQ ? 1 : -1) : 0;
                const float* tb =
                    (kSeveral || near)
                        ? bias + (DQ ? col - x : x - col) - a.q_offset + span.left + kBiasMargin
                        : bias + (low >= span.right ? nbias - 1 : 0);
                const uint64_t scale2 = pair(a.scale2, a.scale2);
                const ulonglong2* qlse =  // two pairs of queries each
                    reinterpret_cast<const ulonglong2*>(stage + 2 * S::kTile) + 8 * half + 4 * c;
                const ulonglong2* qdelta = qlse + kTileRows / 4;
                float p[16], z[16], ds[16];
                uint64_t mass = 0, sum2 = 0;  // sums of p and dS, two lanes of them
                tmem_wait_ld(vs);
                tmem_wait_ld(vp);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  uint64_t shift;  // bias - lse
                  if (DQ && !kSeveral && !kMask) {
                    shift = pair(far + nlse, far + nlse);
                  } else {
                    uint64_t nl;
                    if (DQ) {
                      nl = pair(nlse, nlse);
                    } else {
                      const ulonglong2 four = qlse[k >> 1];
                      nl = k & 1 ? four.y : four.x;
                    }
                    if (kSeveral)
                      shift = add2(DQ ? pair(tb[2 * k], tb[2 * k + 1])
                                      : pair(tb[-2 * k], tb[-2 * k - 1]),
                                   nl);
                    else if (kMask && a.biased)
                      shift = add2(pair(tb[2 * k * step], tb[(2 * k + 1) * step]), nl);
                    else
                      shift = add2(pair(far, far), nl);
                  }
                  unpair(fma2(pair(vs[2 * k], vs[2 * k + 1]), scale2, shift), &p[2 * k],
                         &p[2 * k + 1]);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  p[k] = exp2_approx(p[k]);
                  if (kMask) p[k] = (DQ ? col + k < limit : col + k >= limit) ? p[k] : 0.0f;
                }
                if (DROP && DQ) {
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const uint32_t v[4] = {words[k].x, words[k].y, words[k].z, words[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      keep_pair(v[e], T2, p[8 * k + 2 * e], p[8 * k + 2 * e + 1],
                                &z[8 * k + 2 * e], &z[8 * k + 2 * e + 1]);
                  }
                } else {
#pragma unroll
                  for (int k = 0; k < 16; ++k) z[k] = !DROP || (kept >> k & 1) ? p[k] : 0.0f;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  uint64_t nd;
                  if (DQ) {
                    nd = pair(ndelta, ndelta);
                  } else {
                    const ulonglong2 four = qdelta[k >> 1];
                    nd = k & 1 ? four.y : four.x;
                  }
                  const uint64_t pp = pair(p[2 * k], p[2 * k + 1]);
                  float &d0 = ds[2 * k], &d1 = ds[2 * k + 1];
                  if constexpr (EXACT)
                    unpair(mul2(pair(z[2 * k], z[2 * k + 1]), pair(vp[2 * k], vp[2 * k + 1])), &d0,
                           &d1);
                  else
                    unpair(fma2(pair(z[2 * k], z[2 * k + 1]), pair(vp[2 * k], vp[2 * k + 1]),
                                mul2(pp, nd)),
                           &d0, &d1);
                  if (EXACT || (DQ && !kSeveral)) mass = add2(mass, pp);
                  if (kMask) {
                    const int n = col + 2 * k;
                    d0 = (DQ ? n < limit : n >= limit) ? d0 : 0.0f;
                    d1 = (DQ ? n + 1 < limit : n + 1 >= limit) ? d1 : 0.0f;
                  }
                  if (DQ) sum2 = add2(sum2, pair(d0, d1));
                }
                if (!EXACT) {
                  uint32_t o[8];
                  if (!DQ) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = pack2<T>(z[2 * k], z[2 * k + 1]);
                    tmem_st8(ts + 8 * c, o);
                  }
#pragma unroll
                  for (int k = 0; k < 8; ++k) o[k] = pack2<T>(ds[2 * k], ds[2 * k + 1]);
                  tmem_st8(tp + 8 * c, o);
                }
                if (DQ && a.sum_bufs) {
                  float s0, s1;
                  unpair(sum2, &s0, &s1);
                  const float sum = s0 + s1;
                  eps += sum;
                  if (EXACT) {
                    unpair(mass, &s0, &s1);
                    mass_l += s0 + s1;
                  } else if (!kSeveral && !(kMask && near)) {
                    unpair(mass, &s0, &s1);
                    if (low >= span.right) {
                      far_r += sum;
                      mass_r += s0 + s1;
                    } else {
                      far_l += sum;
                      mass_l += s0 + s1;
                    }
                  } else {
                    // Sums down the diagonals of the 32 x 16 block: a running sum moves one
                    // lane (row) on with every column; what lane 31 then holds is complete.
#pragma unroll
                    for (int k = 1; k < 8; ++k) {  // in two chains, of eight columns
                      add_from_below(&ds[k], ds[k - 1]);
                      add_from_below(&ds[8 + k], ds[7 + k]);
                    }
                    if (lane == 31) {
#pragma unroll
                      for (int k = 0; k < 16; k += 4)
                        *reinterpret_cast<float4*>(bar.carry[warp] + k) =
                            make_float4(ds[k], ds[k + 1], ds[k + 2], ds[k + 3]);
                    }
                    // Eight columns on, the first chain's rows meet the second's; its last
                    // eight rows leave the block.
                    const float first = __shfl_up_sync(0xffffffffu, ds[7], 8);
                    __syncwarp();
                    // of the diagonal of the warp's first row and first column
                    float* to = by_d + warp * ndist + low + 31 + span.left + kSumMargin;
                    if (lane < 15 && lane != 7) to[lane - 31] += bar.carry[warp][lane];
                    __syncwarp();
                    to[15 - lane] += lane < 8 ? ds[15] : ds[15] + first;
                    if (lane >= 24) to[7 - lane] += ds[7];
                    __syncwarp();
                  }
                }
              };
              using Yes = std::true_type;
              using No = std::false_type;
              if (masked)
                weigh(No(), Yes());
              else if (near)
                weigh(Yes(), No());
              else
                weigh(No(), No());
              kept >>= 16;
            }
            if (!ok) break;
            if constexpr (EXACT) {  // the scores have been read: their place and the stage are free
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.empty[st]);
              continue;
            }
            tmem_wait_st();
            if (DQ && keys < a.Lk && c0 + 32 > keys) {
              // Rows of K past the last key have dS = 0, but may hold anything.
              const int live = max(0, keys - c0);  // of the group's 32
              for (int k = threadIdx.x & 127; k < (32 - live) * 8 * (DP / 64); k += 128) {
                const int r = 32 * half + live + (k >> 3) % (32 - live), y = (k >> 3) / (32 - live);
                *reinterpret_cast<uint4*>(stage + y * (kTileRows * 128) + r * 128 + (k & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
              fence_async_shared();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.p_full[slot]);
            if (pending) {
              pending = false;
              finish(k - 1);
            }
          }
          if (a.biased) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.bias_empty[nb & 1]);
            ++nb;
          }
        }
        nt += heads * it.per;
        if (DQ && a.sum_bufs && ok) {
          if constexpr (EXACT) {
            by_d[g * kRows + row] = mass_l;
            by_d[(G + g) * kRows + row] = eps;
          } else {
            float* r = by_d + S::kWarps * ndist + g * kRows + row;
            const float v[5] = {eps, far_l, far_r, mass_l, mass_r};
#pragma unroll
            for (int i = 0; i < 5; ++i) r[i * G * kRows] = v[i];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.sums_full[k % a.sum_bufs]);
        }
      }
      if (ok && pending) finish(k - 1);
      pending = have && !EXACT;
      if (!ok || !have) break;
      __syncwarp();
      if (lane == 0) bar.done[warp] = it;
      __syncwarp();
      have = take(k + 1, it, fetch);
    }
  }
  __syncthreads();
  if (warp == kProducts) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  if (!DQ) grid_wait();  // so that this grid's end is that of all before it
}

int blocks_of(int L) { return (L + kRows - 1) / kRows; }

int exact_tiles(const AttnArgs& a) {
  const bool ragged = a.kv_len && a.Lk > kExactTilesTable * kTileRows;
  return a.dtable && !ragged ? kExactTilesTable : kExactTiles;
}

// The first blocks of 128 queries, those that may have pieces for EXACT: all,
// where an entry may be short; else, with a causal mask, the first queries.
int exact_blocks(const AttnArgs& a) {
  const int most = exact_tiles(a) * kTileRows, blocks = a.Lk ? blocks_of(a.Lq) : 0;
  if (a.Lk <= most || a.kv_len) return blocks;
  if (!a.causal) return 0;
  // block i ends at query min(128 (i + 1), Lq), which sees q_offset keys more
  if (a.Lq + a.q_offset <= most) return blocks;
  return a.q_offset < most ? std::min(blocks, (most - a.q_offset) / kRows) : 0;
}

template <typename T, int DP, bool DQ, bool DROP, bool EXACT>
cudaError_t grad_of(const AttnArgs& a, GradArgs f, cudaStream_t s) {
  using S = GradShape<DP, DQ>;
  const int Lx = DQ ? a.Lq : a.Lk, Hx = DQ ? a.H : a.Hkv;
  f.out1 = DQ ? a.dq : a.dv;
  f.out2 = DQ ? a.dq : a.dk;
  f.blocks = EXACT ? exact_blocks(a) : (Lx + kRows - 1) / kRows;
  f.items = f.blocks * a.B * (f.join ? a.H : Hx);
  f.next += DQ ? 0 : 1;
  constexpr size_t most = 227 * 1024 - 256 - sizeof(GradBars<S::kWarps, S::kStages>);
  size_t bytes = 1024 + S::kBias;
  if (a.biased) {
    const int n = bias_floats(a.rp);
    bytes += 2 * bias_room(n) * sizeof(float);
    if (DQ && !EXACT && f.dtable) {
      // Two buffers, so that the sums of a piece are added up beside the next
      // one; a wide bias may leave room for one.
      const size_t one = S::sum_floats(sum_dists(n)) * sizeof(float);
      f.sum_bufs = bytes + 2 * one <= most ? 2 : 1;
      bytes += f.sum_bufs * one;
    }
  }
  if (EXACT) {
    f.exact_tiles = exact_tiles(a);
    f.sum_bufs = 2;
    bytes += f.sum_bufs * S::kExactFloats * sizeof(float);
  }
  constexpr size_t widest = EXACT ? 2 * S::kExactFloats * sizeof(float)
                                  : S::sum_floats(sum_dists(kBiasMost)) * sizeof(float);
  static_assert(1024 + S::kBias + 8 * bias_room(kBiasMost) + (DQ ? widest : 0) <= most,
                "the widest bias must fit");
  static PerDeviceOnce once;
  cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(k_attn_grad<T, DP, DQ, DROP, EXACT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return launch_behind(k_attn_grad<T, DP, DQ, DROP, EXACT>, dim3(f.items < sms ? f.items : sms),
                       dim3(S::kThreads), bytes, s, f);
}

template <typename T, bool DQ, bool EXACT = false>
cudaError_t grad(const AttnArgs& a, const GradArgs& f, cudaStream_t s) {
  if (a.D <= 64)
    return a.keep.T ? grad_of<T, 64, DQ, true, EXACT>(a, f, s)
                    : grad_of<T, 64, DQ, false, EXACT>(a, f, s);
  return a.keep.T ? grad_of<T, 128, DQ, true, EXACT>(a, f, s)
                  : grad_of<T, 128, DQ, false, EXACT>(a, f, s);
}

constexpr size_t kCounterBytes = 256;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

size_t rows_bytes(const AttnArgs& a) {
  return up256((size_t)a.B * a.H * blocks_of(a.Lq) * kRows * 2 * sizeof(float));
}

size_t partial_bytes(const AttnArgs& a) {
  return a.biased ? up256((size_t)a.B * a.H * blocks_of(a.Lq) * a.rp.num_buckets * sizeof(float))
                  : 0;
}

// Whether dk and dv are worked out for every query head on its own, in fp32,
// and joined by a kernel after: where shared heads leave fewer pieces than the
// card has SMs (152), each as long as its group is large (3 x 517 keys, 2 heads
// shared by 8: backward 66 -> 46 us).
bool splits(const AttnArgs& a) {
  return a.H != a.Hkv && (int64_t)blocks_of(a.Lk) * a.B * a.Hkv < 152;
}

size_t join_bytes(const AttnArgs& a) {
  return splits(a) ? 2 * sizeof(float) * (size_t)a.B * a.H * a.Lk * a.D : 0;
}

// dk and dv: the sums of their group's heads, in order.
struct JoinArgs {
  const float* join;
  int B, H, Hkv, Lk, D;
  Heads dv, dk;
};

template <typename T>
__global__ void __launch_bounds__(256) k_join(const JoinArgs a) {
  grid_wait();
  const int chunks = a.D / 8, group = a.H / a.Hkv;
  int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(t % chunks) * 8;
  t /= chunks;
  const int j = (int)(t % a.Lk);
  t /= a.Lk;
  const int hk = (int)(t % a.Hkv);
  t /= a.Hkv;
  const int b = (int)(t % a.B), which = (int)(t / a.B);
  if (which > 1) return;
  float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int g = 0; g < group; ++g) {
    const float4* p = reinterpret_cast<const float4*>(
        a.join + (((int64_t)(which * a.B + b) * a.H + hk * group + g) * a.Lk + j) * a.D + d);
    const float4 x = p[0], y = p[1];
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += v[i];
  }
  const Heads& out = which ? a.dk : a.dv;
  *reinterpret_cast<uint4*>(static_cast<T*>(out.data) + b * out.b + (int64_t)j * out.l +
                            hk * out.h + d) =
      make_uint4(pack2<T>(s[0], s[1]), pack2<T>(s[2], s[3]), pack2<T>(s[4], s[5]),
                 pack2<T>(s[6], s[7]));
}

template <typename T>
cudaError_t bwd(const AttnArgs& a, cudaStream_t s) {
  GradArgs f{};
  cudaError_t e = attn_error_word(&f.err);
  if (e != cudaSuccess) return e;
  f.B = a.B;
  f.H = a.H;
  f.Hkv = a.Hkv;
  f.D = a.D;
  f.Lq = a.Lq;
  f.Lk = a.Lk;
  f.causal = a.causal;
  f.q_offset = a.q_offset;
  f.biased = a.biased;
  f.scale = a.scale;
  f.scale2 = a.scale * kLog2e;
  f.rp = a.rp;
  f.table = a.table;
  f.kv_len = a.kv_len;
  f.keep = a.keep;
  char* ws = static_cast<char*>(a.workspace);
  f.next = reinterpret_cast<unsigned*>(ws);
  f.rows = reinterpret_cast<float*>(ws + kCounterBytes);
  f.partial = reinterpret_cast<float*>(ws + kCounterBytes + rows_bytes(a));
  f.Lqp = blocks_of(a.Lq) * kRows;
  f.sum_parts = a.B * blocks_of(a.Lq);
  f.dtable = a.dtable;
  // An empty side is never read; its map still needs an address and an extent.
  auto map = [&](CUtensorMap* m, const Heads& t, int L, int heads) {
    return L ? attn_tensor_map(m, t, a.type, a.D, L, heads, a.B, kTileRows)
             : attn_tensor_map(m, a.Lq ? a.q : a.k, a.type, a.D, 1, 1, 1, kTileRows);
  };
  if (a.Lq || a.Lk) {
    e = map(&f.q, a.q, a.Lq, a.H);
    if (e == cudaSuccess) e = map(&f.grad_o, a.grad_o, a.Lq, a.H);
    if (e == cudaSuccess) e = map(&f.k, a.k, a.Lk, a.Hkv);
    if (e == cudaSuccess) e = map(&f.v, a.v, a.Lk, a.Hkv);
    if (e != cudaSuccess) return e;
  }
  RowArgs r{a.B, a.H, a.D, a.Lq, f.Lqp, a.o, a.grad_o, a.lse, 1.0f / a.keep.scale, f.rows, f.next};
  const int64_t blocks = (int64_t)a.B * a.H * blocks_of(a.Lq);
  const unsigned grid_rows = (unsigned)(blocks ? blocks : 1);  // one clears the counters
  if (a.D <= 64)
    k_rows<T, 8><<<grid_rows, kRowThreads, 0, s>>>(r);
  else
    k_rows<T, 16><<<grid_rows, kRowThreads, 0, s>>>(r);
  e = cudaGetLastError();
  if (e == cudaSuccess && a.Lq && exact_blocks(a)) e = grad<T, true, true>(a, f, s);
  if (e == cudaSuccess && a.Lq) e = grad<T, true>(a, f, s);
  if (e != cudaSuccess || !a.Lk) return e;
  if (!a.Lq) f.dtable = nullptr;
  f.behind_dq = a.Lq != 0;
  if (splits(a))
    f.join = reinterpret_cast<float*>(ws + kCounterBytes + rows_bytes(a) + partial_bytes(a));
  e = grad<T, false>(a, f, s);
  if (e != cudaSuccess || !f.join) return e;
  const JoinArgs j{f.join, a.B, a.H, a.Hkv, a.Lk, a.D, a.dv, a.dk};
  const int64_t threads = 2ll * a.B * a.Hkv * a.Lk * (a.D / 8);
  return launch_behind(k_join<T>, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, j);
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a) {
  return kCounterBytes + rows_bytes(a) + partial_bytes(a) + join_bytes(a);
}

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s) {
  if (a.dtable && (a.B == 0 || a.Lq == 0 || a.Lk == 0)) {
    const cudaError_t e = cudaMemsetAsync(a.dtable, 0, (size_t)a.rp.num_buckets * a.H * 2, s);
    if (e != cudaSuccess) return e;
  }
  if (a.B == 0) return cudaSuccess;
  return a.type == OB_TYPE_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<__half>(a, s);
}

}  // namespace ob
