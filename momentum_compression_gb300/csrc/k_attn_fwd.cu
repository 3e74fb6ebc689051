// Attention, forward.
//
// A block takes 256 queries of one head, 128 for each of two warpgroups (a
// thread a query), and walks over the keys in tiles of 64.  One warp issues
// the products on the tensor cores and one the TMA copies:
//   S = Q K^T        128 x 64 in tensor memory, both operands in shared memory
//   P = softmax-to-be of S, dropped and rounded, over S in tensor memory
//   O += P V         P from tensor memory, V as it lies (rows are the sum)
// With head sizes up to 64 two blocks share an SM, and one's products run
// beside the other's arithmetic.  Above, one block fills the SM's tensor
// memory, and a warpgroup's S has two buffers: the scores of the next tile are
// there when it is done with one.
// The softmax is on line: weights are taken relative to a reference m that a
// row raises (with its sum and its O) only when a score passes it by more
// than 2^8, so O is hardly ever touched outside the products.  P is rounded to
// the inputs' type, as the matrix unit wants it; its row sum is of the values
// before that, in fp32.
//
// What bounds it: at d 128 the matrix unit and the softmax beside it, each
// waiting for the other (8192 keys 0.83 ms, 1320 TFLOP/s, 70% of cuBLAS's; 8 x
// 2048 causal 0.15 ms, 910, 48%: the pipe is busy in 43% of the cycles, and
// the start and end of each block are exposed), at d 64 the
// exponentials and the rest of a row's arithmetic (2048 keys 860 TFLOP/s),
// with dropout the drawing of the keep bits, 72 issue cycles of a scheduler
// for 256 pairs (32 x 12 x 512 of d 64 96 us, without dropout 59).
#include <cmath>
#include <type_traits>

#include "attn.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

__device__ unsigned g_attn_error;

constexpr int kRows = 128;      // queries of a warpgroup
constexpr int kGroups = 2;      // warpgroups
constexpr int kCompute = kGroups * 128;
constexpr int kThreads = kCompute + 64;  // and a warp each for products and copies
constexpr int BN = 64;          // keys of a tile
constexpr float kRaise = 8.0f;

struct FwdArgs {
  CUtensorMap q, k, v;
  int B, H, Hkv, D, Lq, Lk, causal, q_offset, biased;
  int parts;  // blocks (a cluster) that share the keys of the same queries
  float scale2;  // scale * log2(e)
  ob_relpos rp;
  const void* table;
  const int32_t* kv_len;
  Keep keep;
  Heads o;
  float* lse;
};

template <int DP>
struct FwdShape {
  static constexpr int kStages = DP == 64 ? 3 : 4;
  static constexpr int kBufs = DP == 64 ? 1 : 2;  // buffers of a warpgroup's S
  static constexpr uint32_t kQ = kRows * DP * 2;  // bytes of one warpgroup's Q
  static constexpr uint32_t kTile = BN * DP * 2;
  // tensor memory: the S, then the O
  static constexpr uint32_t kO = kGroups * kBufs * BN, kAlloc = DP == 64 ? 256 : 512;
  static_assert(kO + kGroups * DP <= kAlloc, "");
  static constexpr uint32_t kBias = kGroups * kQ + 2 * kStages * kTile;  // offset of the bias
  static_assert(kGroups * kRows * DP * 4 <= kBias, "O in fp32 must fit over the operands");
};

struct FwdBars {
  uint64_t q_full, k_full[4], v_full[4], k_empty[4], v_empty[4];
  // By a tile's number modulo 2: with two buffers of S a warpgroup may be a tile
  // ahead of its products, and one barrier's phases would pass each other.
  uint64_t s_full[kGroups][2], p_full[kGroups][2], o_done[kGroups][2];
  uint64_t drain;
  uint32_t tmem;
  uint8_t bucket[kBiasMost];
  float2 ml[kGroups * kRows];  // parts > 1: a row's reference and sum
};

// Where the c-th 16 bytes of a row lie: a warp's rows in different banks.
__device__ __forceinline__ int swap4(int row, int c) { return c ^ (row & 7); }

// The cluster's P parts joined, in order: eight columns of a row a thread, the
// rows spread over the blocks.  os: O of the block's rows, ml: their (m, l).
template <typename T, int DP, int P>
__device__ __forceinline__ void join_parts(const FwdArgs& a, uint32_t os, uint32_t ml, int q0,
                                           int b, int h) {
  const int chunks = a.D / 8, rows = min(kGroups * kRows, a.Lq - q0);
  for (int t = (int)blockIdx.z * kThreads + threadIdx.x; t < rows * chunks; t += P * kThreads) {
    const int r = t / chunks, c = t % chunks;
    float2 of[P];
    float4 v[P][2];
#pragma unroll
    for (int p = 0; p < P; ++p) of[p] = cluster_ld2(ml + 8 * r, p);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        v[p][x] = cluster_ld4(os + 16 * (r * (DP / 4) + swap4(r, 2 * c + x)), p);
    float m = -INFINITY, l = 0.0f, o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < P; ++p) m = fmaxf(m, of[p].x);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (of[p].y == 0.0f) continue;  // no key with weight: its O may not be there
      const float w = of[p].x == -INFINITY ? 1.0f : exp2_approx(of[p].x - m);  // no reference: NaN
      l = __fmaf_rn(of[p].y, w, l);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        o[4 * x] = __fmaf_rn(v[p][x].x, w, o[4 * x]);
        o[4 * x + 1] = __fmaf_rn(v[p][x].y, w, o[4 * x + 1]);
        o[4 * x + 2] = __fmaf_rn(v[p][x].z, w, o[4 * x + 2]);
        o[4 * x + 3] = __fmaf_rn(v[p][x].w, w, o[4 * x + 3]);
      }
    }
    const float inv = l > 0.0f || l != l ? a.keep.scale / l : 0.0f;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (inv != 0.0f)
      u = make_uint4(pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv),
                     pack2<T>(o[4] * inv, o[5] * inv), pack2<T>(o[6] * inv, o[7] * inv));
    *reinterpret_cast<uint4*>(static_cast<T*>(a.o.data) + b * a.o.b + (int64_t)(q0 + r) * a.o.l +
                              h * a.o.h + 8 * c) = u;
    if (a.lse && c == 0)
      a.lse[((size_t)b * a.H + h) * a.Lq + q0 + r] =
          l != 0.0f ? __fmaf_rn(m, kLn2, logf(l)) : -INFINITY;
  }
}

template <typename T, int DP, bool DROP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1)
    k_attn_fwd(const __grid_constant__ FwdArgs a) {
  using S = FwdShape<DP>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  // The next columns' scores on their way while these are worked on, where the
  // registers last for it.
  constexpr bool kAhead = DP > 64 || !DROP;
  extern __shared__ uint8_t raw[];
  __shared__ FwdBars bar;
  uint8_t* smem = align_shared(raw);
  float* bias = reinterpret_cast<float*>(smem + S::kBias);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hkv);
  // The last queries see the most keys: they start first, those of all heads.
  const int q0 = ((int)gridDim.y - 1 - (int)blockIdx.y) * (kGroups * kRows);
  const int keys = key_count(a, b);
  int tiles[kGroups], most = 0;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int qg = q0 + g * kRows;
    int n = keys;
    if (a.causal) n = min(n, min(qg + kRows, a.Lq) + a.q_offset);
    tiles[g] = qg < a.Lq && n > 0 ? (n + BN - 1) / BN : 0;
    most = max(most, tiles[g]);
  }
  // Of these tiles the block takes `per` from t0 on.
  const int per = SPLIT ? (most + a.parts - 1) / a.parts : most;
  const int t0 = SPLIT ? (int)blockIdx.z * per : 0;
  if (SPLIT) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) tiles[g] = max(0, min(tiles[g] - t0, per));
    most = max(0, min(most - t0, per));
  }

  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, 1);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int g = 0; g < kGroups; ++g) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bar.s_full[g][i], 1);
        mbar_init(&bar.p_full[g][i], kRows / 32);
        mbar_init(&bar.o_done[g][i], 1);
      }
    }
    mbar_init(&bar.drain, 1);
    fence_barrier_init();
  }
  if (warp == kCompute / 32) tmem_alloc(&bar.tmem, S::kAlloc);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  if (warp == kCompute / 32 + 1) {
    // ----- copies --------------------------------------------------------
    if (most > 0) {
      if (lane == 0) {
        uint32_t groups = 0;
        for (int g = 0; g < kGroups; ++g) groups += tiles[g] > 0;
        mbar_arrive_expect_tx(&bar.q_full, groups * S::kQ);
        for (int g = 0; g < kGroups; ++g)
          if (tiles[g] > 0)
            for (int x = 0; x < DP / 64; ++x)
              tma_load4(smem + g * S::kQ + x * (kRows * 128), &a.q, 64 * x, q0 + g * kRows, h, b,
                        &bar.q_full);
      }
      bool ok = true;
      int n = 0, nv = 0;  // tiles of K and V asked for
      for (; n < most; ++n, ++nv) {
        const int st = n % S::kStages;
        const uint32_t par = (n / S::kStages + 1) & 1;
        uint8_t* kt = smem + kGroups * S::kQ + 2 * st * S::kTile;
        if (n >= S::kStages) ok = warp_wait(&bar.k_empty[st], par, &g_attn_error, kErrWaitEmpty);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.k_full[st], S::kTile);
          for (int x = 0; x < DP / 64; ++x)
            tma_load4(kt + x * (BN * 128), &a.k, 64 * x, (t0 + n) * BN, hk, b, &bar.k_full[st]);
        }
        if (n >= S::kStages) ok = warp_wait(&bar.v_empty[st], par, &g_attn_error, kErrWaitEmpty);
        if (!ok) {
          ++n;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&bar.v_full[st], S::kTile);
          for (int x = 0; x < DP / 64; ++x)
            tma_load4(kt + S::kTile + x * (BN * 128), &a.v, 64 * x, (t0 + n) * BN, hk, b,
                      &bar.v_full[st]);
        }
      }
      if (!ok) {  // a wait ran out: let what is in flight land before the block ends
        mbar_wait(&bar.q_full, 0, &g_attn_error, kErrDrain);
        for (int i = max(0, n - S::kStages); i < n; ++i)
          mbar_wait(&bar.k_full[i % S::kStages], (i / S::kStages) & 1, &g_attn_error, kErrDrain);
        for (int i = max(0, nv - S::kStages); i < nv; ++i)
          mbar_wait(&bar.v_full[i % S::kStages], (i / S::kStages) & 1, &g_attn_error, kErrDrain);
      }
    }
  } else if (warp == kCompute / 32) {
    // ----- products ------------------------------------------------------
    if (most > 0) {
      constexpr uint32_t kShapeS = mma_shape(kBf16, BN, false);
      constexpr uint32_t kShapeO = mma_shape(kBf16, DP, true);
      const uint32_t leader = elect_lane();
      const uint32_t qs = smem_u32(smem), kv = qs + kGroups * S::kQ;
      const uint64_t q_desc = desc_k(qs), k_desc = desc_k(kv),
                     v_desc = desc_mn(kv + S::kTile, BN * 128);
      const int ksteps = (a.D + 15) / 16;
      bool ok = warp_wait(&bar.q_full, 0, &g_attn_error);
      int kst = 0, kpar = 0, kn = 0;  // stage, phase and number of the next tile of K
      // S of tile kn for both groups; its buffer's P has been issued to O.
      auto scores = [&](int g) {
        const uint64_t qd = q_desc + (uint32_t)g * (S::kQ >> 4);
        const uint64_t kd = k_desc + (uint32_t)kst * (2 * S::kTile >> 4);
        const uint32_t d = tmem + (g * S::kBufs + kn % S::kBufs) * BN;
#pragma unroll
        for (int s = 0; s < DP / 16; ++s)
          if (s < ksteps)
            mma_ss(leader, d, qd + (((s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4),
                   kd + (((s >> 2) * (BN * 128) + (s & 3) * 32) >> 4), kShapeS, s > 0);
        mma_commit(leader, &bar.s_full[g][kn & 1]);
      };
      auto next_k = [&] {  // that tile of K is issued for both
        // Only where a later copy waits for it: nothing may arrive after the block's end.
        if (kn + S::kStages < most) mma_commit(leader, &bar.k_empty[kst]);
        ++kn;
        if (++kst == S::kStages) kst = 0, kpar ^= 1;
      };
      for (int i = 0; ok && i < S::kBufs && i < most; ++i) {
        ok = warp_wait(&bar.k_full[kst], kpar, &g_attn_error);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          if (kn < tiles[g]) scores(g);
        next_k();
      }
      int st = 0, par = 0;  // of tile n of V
      for (int n = 0; ok && n < most; ++n) {
        ok = warp_wait(&bar.v_full[st], par, &g_attn_error);
        if (ok && kn < most) ok = warp_wait(&bar.k_full[kst], kpar, &g_attn_error);
        const uint64_t vd = v_desc + (uint32_t)st * (2 * S::kTile >> 4);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          if (!ok || n >= tiles[g]) continue;
          ok = warp_wait(&bar.p_full[g][n & 1], (n >> 1) & 1, &g_attn_error);
          if (!ok) continue;
          tc_fence_after();
          const uint32_t p = tmem + (g * S::kBufs + n % S::kBufs) * BN;
#pragma unroll
          for (int s = 0; s < BN / 16; ++s)
            mma_ts(leader, tmem + S::kO + g * DP, p + s * 8, vd + s * (2048 >> 4), kShapeO,
                   n > 0 || s > 0);
          mma_commit(leader, &bar.o_done[g][n & 1]);
          if (kn < tiles[g]) scores(g);
        }
        if (ok && n + S::kStages < most) mma_commit(leader, &bar.v_empty[st]);
        if (ok && kn < most) next_k();
        if (++st == S::kStages) st = 0, par ^= 1;
      }
      if (!ok) {
        mma_commit(leader, &bar.drain);
        mbar_wait(&bar.drain, 0, &g_attn_error, kErrDrain);
      }
    }
  } else {
    // ----- softmax: a thread a query -------------------------------------
    if (a.biased) {  // while the first copies are on their way
      stage_buckets(bar.bucket, a.rp, threadIdx.x, kCompute);
      named_sync(1, kCompute);
      stage_bias(bias, bar.bucket, bias_floats(a.rp), static_cast<const T*>(a.table), a.H, h,
                 threadIdx.x, kCompute);
      named_sync(1, kCompute);
    }
    const int g = warp >> 2, mine = g ? tiles[1] : tiles[0];
    const int row = (warp & 3) * 32 + lane;
    const int i = q0 + g * kRows + row;
    const int wi = q0 + g * kRows + (warp & 3) * 32;  // the warp's first query
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + S::kO + g * DP;
    const int limit = a.causal ? min(keys, i + a.q_offset + 1) : keys;  // keys of this row
    const int warp_limit = a.causal ? min(keys, wi + a.q_offset + 1) : keys;  // of the first
    const uint32_t T2 = a.keep.T * 0x10001u;
    const uint64_t call0 = ((uint64_t)bh * a.Lq + i) * (uint32_t)((a.Lk + 7) / 8);
    const BiasSpan span = a.biased ? bias_span(a.rp) : BiasSpan{0, 0};
    const int nbias = a.biased ? bias_floats(a.rp) : 0;
    const float far_left = a.biased ? bias[0] : 0.0f, far_right = a.biased ? bias[nbias - 1] : 0.0f;
    const uint64_t scale2 = pair(a.scale2, a.scale2);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;

    for (int n = 0; n < mine; ++n) {
      const uint32_t ts = tmem + lanes + (g * S::kBufs + n % S::kBufs) * BN;
      const int j0 = (t0 + n) * BN;
      // The keep bits do not wait for the scores: as masks of the packed weights.
      uint32_t p[BN / 2];
      auto draw = [&] {
#pragma unroll
        for (int k = 0; k < BN / 8; k += 4) {
          uint4 w[4];
          keep_words_n(a.keep, call0 + (uint32_t)((t0 + n) * (BN / 8) + k), 1, w);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            p[4 * (k + q)] = keep_mask2(w[q].x, T2);
            p[4 * (k + q) + 1] = keep_mask2(w[q].y, T2);
            p[4 * (k + q) + 2] = keep_mask2(w[q].z, T2);
            p[4 * (k + q) + 3] = keep_mask2(w[q].w, T2);
          }
        }
      };
      if (DROP) draw();
      ok = warp_wait(&bar.s_full[g][n & 1], (n >> 1) & 1, &g_attn_error);
      if (!ok) break;
      tc_fence_after();
      // Distances of the warp's rows and the tile's columns: [low, low + 94].
      const int low = j0 - wi - 31 - a.q_offset;
      const bool near = a.biased && low + 94 > -span.left && low < span.right;
      const float far = low >= span.right ? far_right : far_left;
      const bool masked = j0 + BN > warp_limit;

      // The largest score of the tile, times log2(e).
      auto peak = [&] {
        const int step = near ? 1 : 0;
        const float* t = near ? bias + (j0 - i - a.q_offset) + span.left + kBiasMargin
                              : bias + (low >= span.right ? nbias - 1 : 0);
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
          uint32_t v[16];
          tmem_ld16(v, ts + c);
          tmem_wait_ld(v);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float s = __uint_as_float(v[k]);
            float x = a.biased ? __fmaf_rn(s, a.scale2, t[(c + k) * step]) : s * a.scale2;
            x = j0 + c + k < limit ? x : -INFINITY;
            top = fmaxf(top, x);
          }
        }
        return top;
      };
      float sum, top;  // top: relative to base
      // The weights relative to base, into p (dropped ones as zero), their sum and
      // their largest score.  Branch-free inside, for the scheduler's sake: a body
      // each for tiles of one bias value, tiles across several, and tiles with
      // masked pairs (of either kind).
      auto weigh = [&](auto several_t, auto mask_t, float base) {
        constexpr bool kSeveral = decltype(several_t)::value, kMask = decltype(mask_t)::value;
        const int step = kSeveral || near ? 1 : 0;
        const float* t = kSeveral || near
                             ? bias + (j0 - i - a.q_offset) + span.left + kBiasMargin
                             : bias + (low >= span.right ? nbias - 1 : 0);
        const uint64_t less = pair(-base, -base);
        const float f = (a.biased ? far : 0.0f) - base;
        uint64_t sum2 = 0;
        top = -INFINITY;
        uint32_t r[kAhead ? 2 : 1][16];
        if (kAhead) tmem_ld16(r[0], ts);
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) {  // 16 columns
          uint32_t(&v)[16] = r[kAhead ? c & 1 : 0];
          if (!kAhead) tmem_ld16(v, ts + 16 * c);
          tmem_wait_ld(v);
          if (kAhead && c + 1 < BN / 16) tmem_ld16(r[~c & 1], ts + 16 * (c + 1));
          float x[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int n0 = 16 * c + 2 * k;
            uint64_t shift;  // bias - base
            if (kSeveral)
              shift = add2(pair(t[n0], t[n0 + 1]), less);
            else if (kMask && a.biased)
              shift = add2(pair(t[n0 * step], t[(n0 + 1) * step]), less);
            else
              shift = pair(f, f);
            unpair(fma2(pair(v[2 * k], v[2 * k + 1]), scale2, shift), &x[2 * k], &x[2 * k + 1]);
            if (kMask) {
              x[2 * k] = j0 + n0 < limit ? x[2 * k] : -INFINITY;
              x[2 * k + 1] = j0 + n0 + 1 < limit ? x[2 * k + 1] : -INFINITY;
            }
            top = fmaxf(top, fmaxf(x[2 * k], x[2 * k + 1]));
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[2 * k] = exp2_approx(x[2 * k]);
            x[2 * k + 1] = exp2_approx(x[2 * k + 1]);
            sum2 = add2(sum2, pair(x[2 * k], x[2 * k + 1]));
            const uint32_t w = pack2<T>(x[2 * k], x[2 * k + 1]);
            p[8 * c + k] = DROP ? p[8 * c + k] & w : w;
          }
        }
        float s0, s1;
        unpair(sum2, &s0, &s1);
        sum = s0 + s1;
      };
      using Yes = std::true_type;
      using No = std::false_type;
      // The first tile is looked over for its maximum; the others are taken
      // relative to m at once, and again in the rare case that m is passed.
      if (n == 0) m = peak();
#pragma unroll 1
      for (int pass = 0;; ++pass) {
        const float base = m == -INFINITY ? 0.0f : m;
        if (masked)
          weigh(No(), Yes(), base);
        else if (near)
          weigh(Yes(), No(), base);
        else
          weigh(No(), No(), base);
        const bool over = m == -INFINITY ? top > -INFINITY : top > kRaise;
        if (pass == 1 || !__any_sync(0xffffffffu, over)) break;
        const float up = fmaxf(m, base + top);
        const float less = m == -INFINITY ? 0.0f : exp2_approx(m - up);
        m = up;
        l *= less;
        if (n > 0) {
          ok = warp_wait(&bar.o_done[g][(n - 1) & 1], ((n - 1) >> 1) & 1, &g_attn_error);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < DP; c += 16) {
            uint32_t o[16];
            tmem_ld16(o, to + c);
            tmem_wait_ld(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * less);
            tmem_st16(to + c, o);
          }
        }
        if (DROP) draw();
      }
      if (!ok) break;
      l += sum;
#pragma unroll
      for (int c = 0; c < BN / 32; ++c) tmem_st16(ts + 16 * c, p + 16 * c);
      tmem_wait_st();
      if (keys < a.Lk && j0 + BN > keys) {
        // Rows of V past the last key have weight zero, but may hold anything.
        const int st = n % S::kStages;
        ok = warp_wait(&bar.v_full[st], (n / S::kStages) & 1, &g_attn_error);
        if (!ok) break;
        uint8_t* vt = smem + kGroups * S::kQ + (2 * st + 1) * S::kTile;
        const int from = keys - j0;  // > 0: the tile holds a key
        for (int t = threadIdx.x & 127; t < (BN - from) * 8 * (DP / 64); t += 128) {
          const int r = from + (t >> 3) % (BN - from), x = (t >> 3) / (BN - from);
          *reinterpret_cast<uint4*>(vt + x * (BN * 128) + r * 128 + (t & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_full[g][n & 1]);
    }
    if (ok && mine > 0)
      ok = warp_wait(&bar.o_done[g][(mine - 1) & 1], ((mine - 1) >> 1) & 1, &g_attn_error);
    tc_fence_after();
    if constexpr (SPLIT) {
      // ----- m, l and O for the cluster, over the operands ----------------
      named_sync(1, kCompute);  // both groups' products have read them
      float4* own = reinterpret_cast<float4*>(smem) + (g * kRows + row) * (DP / 4);
      bar.ml[g * kRows + row] = make_float2(m, l);
      if (ok && mine > 0) {  // the same for the whole warp, as its loads want it
#pragma unroll 1
        for (int c = 0; c < DP / 16; ++c) {
          uint32_t r[16];
          tmem_ld16(r, to + 16 * c);
          tmem_wait_ld(r);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            own[swap4(row, 4 * c + k)] =
                make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]),
                            __uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
        }
      }
    } else {
      // ----- o = O / l -------------------------------------------------------
      const float inv = l > 0.0f || l != l ? a.keep.scale / l : 0.0f;
      T* out = static_cast<T*>(a.o.data) + b * a.o.b + (int64_t)i * a.o.l + h * a.o.h;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        uint32_t r[32];
        if (mine > 0) {
          tmem_ld32(r, to + 32 * c);
          tmem_wait_ld(r);
        }
        if (i < a.Lq) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (32 * c + 8 * k >= a.D) break;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (inv != 0.0f) {
              uint32_t* u = &w.x;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                u[e] = pack2<T>(__uint_as_float(r[8 * k + 2 * e]) * inv,
                                __uint_as_float(r[8 * k + 2 * e + 1]) * inv);
            }
            *reinterpret_cast<uint4*>(out + 32 * c + 8 * k) = w;
          }
        }
      }
      if (a.lse && i < a.Lq)
        a.lse[(size_t)bh * a.Lq + i] = l != 0.0f ? __fmaf_rn(m, kLn2, logf(l)) : -INFINITY;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kCompute / 32) {
    tc_fence_after();
    tmem_free(tmem, S::kAlloc);
  }
  if constexpr (SPLIT) {
    cluster_sync();
    auto join = [&](auto parts) {
      join_parts<T, DP, decltype(parts)::value>(a, smem_u32(smem), smem_u32(bar.ml), q0, b, h);
    };
    if (a.parts == 2)
      join(std::integral_constant<int, 2>());
    else if (a.parts == 4)
      join(std::integral_constant<int, 4>());
    else
      join(std::integral_constant<int, 8>());
    cluster_sync();  // the others may still read
  }
}

// A launch whose blocks of the same x and y are a cluster.
struct Clusters {
  cudaLaunchConfig_t launch{};
  cudaLaunchAttribute at{};
  Clusters(dim3 grid, int parts, size_t smem, cudaStream_t s) {
    launch.gridDim = grid;
    launch.blockDim = dim3(kThreads);
    launch.dynamicSmemBytes = smem;
    launch.stream = s;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = at.val.clusterDim.y = 1;
    at.val.clusterDim.z = parts;
    launch.attrs = &at;
    launch.numAttrs = 1;
  }
  Clusters(const Clusters&) = delete;  // launch points into it
};

template <typename T, int DP, bool DROP>
cudaError_t fwd(const AttnArgs& a, cudaStream_t s) {
  using S = FwdShape<DP>;
  FwdArgs f{};
  cudaError_t e = attn_tensor_map(&f.q, a.q, a.type, a.D, a.Lq, a.H, a.B, kRows);
  // Without keys nothing is read through these; the map still needs an address.
  if (e == cudaSuccess)
    e = attn_tensor_map(&f.k, a.Lk ? a.k : a.q, a.type, a.D, a.Lk ? a.Lk : 1, a.Lk ? a.Hkv : 1,
                        a.Lk ? a.B : 1, BN);
  if (e == cudaSuccess)
    e = attn_tensor_map(&f.v, a.Lk ? a.v : a.q, a.type, a.D, a.Lk ? a.Lk : 1, a.Lk ? a.Hkv : 1,
                        a.Lk ? a.B : 1, BN);
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
  f.scale2 = a.scale * kLog2e;
  f.rp = a.rp;
  f.table = a.table;
  f.kv_len = a.kv_len;
  f.keep = a.keep;
  f.o = a.o;
  f.lse = a.lse;
  const size_t bytes = 1024 + S::kBias + (a.biased ? bias_floats(a.rp) * sizeof(float) : 0);
  constexpr int most = 1024 + S::kBias + kBiasMostBytes;
  // How many clusters of 2, 4 and 8 blocks the card holds at a time.
  static PerDeviceOnce once;
  static int rooms[64][3];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int(&room)[3] = rooms[dev & 63];
  e = once.run([&] {
    cudaError_t r = cudaFuncSetAttribute(k_attn_fwd<T, DP, DROP, false>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(k_attn_fwd<T, DP, DROP, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    for (int i = 0; i < 3 && r == cudaSuccess; ++i) {
      Clusters c(dim3(1, 1, 2 << i), 2 << i, most, nullptr);
      r = cudaOccupancyMaxActiveClusters(&room[i], k_attn_fwd<T, DP, DROP, true>, &c.launch);
    }
    return r;
  });
  if (e != cudaSuccess) return e;
  // Where the card has room for more blocks, up to eight share the keys of the
  // same queries, as a cluster that joins its parts through shared memory (one
  // query, 12 heads of 64, 8192 keys: 104 -> 19 us).  Joining costs 2 to 4 us, a
  // tile 0.6 us, with dropout 1.4: each keeps six tiles, with dropout three
  // (3 x 8 x 333 x 517 of d 80, nine tiles in two parts: 19.2 -> 17.6 us with
  // dropout, but 12.0 -> 13.3 without).
  const int blocks = (a.Lq + kGroups * kRows - 1) / (kGroups * kRows);
  const int tiles = (a.Lk + BN - 1) / BN, least = DROP ? 3 : 6;
  f.parts = 1;
  for (int i = 0; i < 3; ++i)
    if ((int64_t)a.B * a.H * blocks <= room[i] && tiles >= least * (2 << i)) f.parts = 2 << i;
  const dim3 grid(a.B * a.H, blocks, f.parts);
  if (f.parts == 1) {
    k_attn_fwd<T, DP, DROP, false><<<grid, kThreads, bytes, s>>>(f);
    return cudaGetLastError();
  }
  Clusters c(grid, f.parts, bytes, s);
  return cudaLaunchKernelEx(&c.launch, k_attn_fwd<T, DP, DROP, true>, f);
}

}  // namespace

cudaError_t attn_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attn_error);
}

cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t s) {
  auto by_type = [&](auto zero) {
    using T = decltype(zero);
    if (a.D <= 64)
      return a.keep.T ? fwd<T, 64, true>(a, s) : fwd<T, 64, false>(a, s);
    return a.keep.T ? fwd<T, 128, true>(a, s) : fwd<T, 128, false>(a, s);
  };
  return a.type == OB_TYPE_BF16 ? by_type(__nv_bfloat16()) : by_type(__half());
}

}  // namespace ob
