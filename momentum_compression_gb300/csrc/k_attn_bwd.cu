// Attention, backward.
//
// Three kernels.  k_rows: lse and rowsum(do o) of every query.  k_attn_grad
// twice: for 128 queries at a time over the keys (dq and the bias table's
// sums), and for 128 keys at a time over the queries of the heads that share
// them (dk, dv).  Both recompute S and dP on the tensor cores and need no
// atomics: seven products instead of the five of a single pass, for results
// that are the same bits on every run.
//
// A block holds its 128 rows X, Y in shared memory (q, do or k, v) and walks
// over tiles of 64 of the other side, U, W.  With a thread a row:
//   S = X U^T, dP = Y W^T   128 x 64 each in tensor memory
//   Z, dS                   from them in registers, rounded over S and dP
//   acc1 += Z W (dv), acc2 += dS U (dq or dk)    first operand from tensor memory
// The warpgroups of a block take turns over the tiles, so one's arithmetic
// runs beside another's products.
#include <cmath>
#include <type_traits>

#include "attn.cuh"
#include "ob_internal.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kRows = 128;  // rows of X, Y
constexpr int kTileRows = 64;
constexpr int kRowsPerBlock = 16;  // of k_rows

struct GradArgs {
  CUtensorMap x, y, u, w;
  int B, H, Hkv, D, Lq, Lk, causal, q_offset, biased;
  float scale, scale2;  // scale2 = scale * log2(e)
  ob_relpos rp;
  const void* table;
  const int32_t* kv_len;
  Keep keep;
  float* rows;     // of each tile of 64 queries: 64 times -lse * log2(e) (-inf: no weight),
                   // then 64 times -rowsum(do o) / keep.scale
  int Lqp;
  Heads out1, out2;  // dq: out2 = dq; dkv: out1 = dv, out2 = dk
  float* partial;    // [H][B * blocks][num_buckets], or null
  unsigned* err;
};

struct RowArgs {
  int B, H, D, Lq, Lqp;
  Heads o, grad_o;
  const float* lse;
  float inv_keep;
  float* rows;
};

// ---------------------------------------------------------------------------
// -lse and -rowsum(do o): 16 lanes a row.  Rows past Lq and rows without keys
// get -lse = -inf, which makes every weight exp2(s - lse) zero.
// ---------------------------------------------------------------------------

// Where query i of head bh has the first of its two values; the second is
// kTileRows further.
__device__ __forceinline__ int64_t row_at(int bh, int Lqp, int i) {
  return (int64_t)bh * Lqp * 2 + (int64_t)(i / kTileRows) * (2 * kTileRows) + i % kTileRows;
}

template <typename T>
__global__ void __launch_bounds__(16 * kRowsPerBlock) k_rows(const RowArgs a) {
  const int l = threadIdx.x & 15;
  const int64_t at = (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 4);
  const int bh = (int)(at / a.Lqp), i = (int)(at % a.Lqp), b = bh / a.H, h = bh % a.H;
  if (bh >= a.B * a.H) return;
  float sum = 0.0f;
  if (i < a.Lq && 8 * l < a.D) {
    const uint4 x = *reinterpret_cast<const uint4*>(
        static_cast<const T*>(a.o.data) + b * a.o.b + (int64_t)i * a.o.l + h * a.o.h + 8 * l);
    const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.grad_o.data) +
                                                    b * a.grad_o.b + (int64_t)i * a.grad_o.l +
                                                    h * a.grad_o.h + 8 * l);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack2<T>(xs[k]), g = unpack2<T>(ys[k]);
      sum = __fmaf_rn(f.x, g.x, sum);
      sum = __fmaf_rn(f.y, g.y, sum);
    }
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (l == 0) {
    float nlse = -INFINITY;
    if (i < a.Lq) {
      const float x = a.lse[(int64_t)bh * a.Lq + i];
      if (x != -INFINITY) nlse = -x * kLog2e;
    }
    float* to = a.rows + row_at(bh, a.Lqp, i);
    to[0] = nlse;
    to[kTileRows] = nlse == -INFINITY ? 0.0f : -sum * a.inv_keep;
  }
}

// ---------------------------------------------------------------------------
// The gradients
// ---------------------------------------------------------------------------

template <int DP, bool DQ>
struct GradShape {
  static constexpr int kGroups = DP == 64 ? 3 : 2;
  static constexpr int kStages = DP == 64 ? 5 : 3;
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = 128 * kGroups + 64;
  static constexpr uint32_t kX = kRows * DP * 2;
  static constexpr uint32_t kTile = kTileRows * DP * 2;
  static constexpr uint32_t kStage = 2 * kTile + (DQ ? 0 : 1024);  // U, W and the queries' rows
  static constexpr uint32_t kBias = 2 * kX + kStages * kStage;     // offset of the bias
  // tensor memory: S and dP of each group, the accumulators
  static constexpr uint32_t kAcc = 128 * kGroups;
};

template <int G, int S>
struct GradBars {
  uint64_t x_full, full[S], empty[S], s_full[G], p_full[G], done;
  uint32_t tmem;
  int dead;
  int first[OB_RELPOS_MAX_SIDE];
  float eps[G][kRows];        // sums of a row's dS
  float far[4 * G][2];        // the warps' sums over the far buckets
  float carry[4 * G][32];
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, kErrWaitFull));
}

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

// Keep bits of 32 queries for the thread's key, from calls that hold eight
// keys of one query: lane l draws the queries 8 k + l % 8 (call0 of k = 0, a
// query further every `step` calls) for the eight keys of its eight lanes,
// and an 8 x 8 transposition of bits among those lanes turns query numbers
// into bit numbers.  Bit r: query r.
__device__ __forceinline__ uint32_t keep_column(const Keep& keep, uint64_t call0, uint64_t step,
                                                int lane) {
  uint32_t x = 0, y = 0;  // queries 8 k + l % 8 for k = 0, 1 and for k = 2, 3
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint4 w = keep_words(keep, call0 + (uint64_t)(8 * k) * step);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t& to = k < 2 ? x : y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      to |= keep_mask2(u[e], keep.T * 0x10001u) & (0x00020001u << (2 * e + 8 * (k & 1)));
    }
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

template <typename T, int DP, bool DQ, bool DROP>
__global__ void __launch_bounds__(GradShape<DP, DQ>::kThreads, 1)
    k_attn_grad(const __grid_constant__ GradArgs a) {
  using S = GradShape<DP, DQ>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int G = S::kGroups, kProducts = 4 * G, kCopies = 4 * G + 1;
  extern __shared__ uint8_t raw[];
  __shared__ GradBars<G, S::kStages> bar;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
  float* bias = reinterpret_cast<float*>(smem + S::kBias);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const BiasSpan span = a.biased ? bias_span(a.rp) : BiasSpan{0, 0};
  const int nbias = a.biased ? bias_floats(a.rp) : 0;
  const bool sums = DQ && a.partial;
  float* by_d = bias + nbias;  // the warps' sums by distance, nbias each

  // DQ: x0 is a query of head h.  Else a key of head hk, and the tiles run over
  // the queries from `from` on of the heads h0 .. h0 + heads - 1.
  const int group = a.H / a.Hkv;
  const int b = blockIdx.y / (DQ ? a.H : a.Hkv), hx = blockIdx.y % (DQ ? a.H : a.Hkv);
  const int h0 = DQ ? hx : hx * group, hk = DQ ? hx / group : hx, heads = DQ ? 1 : group;
  const int keys = key_count(a.kv_len, a.Lk, b);
  // Causal: the last queries see the most keys, the first keys the most queries.
  const int x0 = (DQ ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x) * kRows;
  int from = 0, per;  // tiles of a head: from, ..., from + per - 1
  if (DQ) {
    int n = keys;
    if (a.causal) n = min(n, min(x0 + kRows, a.Lq) + a.q_offset);
    per = n > 0 ? (n + kTileRows - 1) / kTileRows : 0;
  } else {
    if (a.causal) from = max(0, x0 - a.q_offset) / kTileRows;
    per = x0 < keys ? max(0, (a.Lq + kTileRows - 1) / kTileRows - from) : 0;
  }
  const int total = heads * per;

  if (threadIdx.x == 0) {
    mbar_init(&bar.x_full, 1);
    mbar_init(&bar.done, 1);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int g = 0; g < G; ++g) {
      mbar_init(&bar.s_full[g], 1);
      mbar_init(&bar.p_full[g], 128);
    }
    bar.dead = 0;
    fence_barrier_init();
  }
  if (warp == kProducts) tmem_alloc(&bar.tmem, 512);
  if (a.biased) {
    for (int i = threadIdx.x; i < a.rp.side; i += S::kThreads) bar.first[i] = a.rp.first[i];
    if (sums)
      for (int i = threadIdx.x; i < S::kWarps * nbias; i += S::kThreads) by_d[i] = 0.0f;
    __syncthreads();
    if (DQ)
      stage_bias(bias, a.rp, bar.first, static_cast<const T*>(a.table), a.H, h0, threadIdx.x,
                 S::kThreads);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  volatile int* dead = &bar.dead;

  if (warp == kCopies) {
    // ----- copies --------------------------------------------------------
    if (lane == 0 && total > 0) {
      mbar_arrive_expect_tx(&bar.x_full, 2 * S::kX);
      for (int x = 0; x < DP / 64; ++x) {
        tma_load4(smem + x * (kRows * 128), &a.x, 64 * x, x0, hx, b, &bar.x_full);
        tma_load4(smem + S::kX + x * (kRows * 128), &a.y, 64 * x, x0, hx, b, &bar.x_full);
      }
      int t = 0;
      for (; t < total; ++t) {
        const int st = t % S::kStages;
        if (t >= S::kStages &&
            (!mbar_wait(&bar.empty[st], (t / S::kStages + 1) & 1, a.err, kErrWaitEmpty) || *dead))
          break;
        uint8_t* to = smem + 2 * S::kX + st * S::kStage;
        const int r = (from + t % per) * kTileRows, hu = DQ ? hk : h0 + t / per;
        mbar_arrive_expect_tx(&bar.full[st], 2 * S::kTile + (DQ ? 0 : kTileRows * 8));
        for (int x = 0; x < DP / 64; ++x) {
          tma_load4(to + x * (kTileRows * 128), &a.u, 64 * x, r, hu, b, &bar.full[st]);
          tma_load4(to + S::kTile + x * (kTileRows * 128), &a.w, 64 * x, r, hu, b, &bar.full[st]);
        }
        if (!DQ)
          bulk_g2s(to + 2 * S::kTile, a.rows + row_at(b * a.H + hu, a.Lqp, r), kTileRows * 8,
                   &bar.full[st]);
      }
      if (t < total) {  // a wait ran out: let what is in flight land before the block ends
        *dead = 1;
        mbar_wait(&bar.x_full, 0, a.err, kErrDrain);
        for (int i = max(0, t - S::kStages); i < t; ++i)
          mbar_wait(&bar.full[i % S::kStages], (i / S::kStages) & 1, a.err, kErrDrain);
      }
    }
  } else if (warp == kProducts) {
    // ----- products ------------------------------------------------------
    if (total > 0) {
      constexpr uint32_t kShapeS = mma_shape(kBf16, kTileRows, false);
      constexpr uint32_t kShapeA = mma_shape(kBf16, DP, true);
      const uint32_t leader = elect_lane();
      const uint32_t xs = smem_u32(smem), us = xs + 2 * S::kX;
      const uint64_t x_desc = desc_k(xs), u_desc = desc_k(us),
                     u_rows = desc_mn(us, kTileRows * 128);
      const int ksteps = (a.D + 15) / 16;
      bool ok = warp_wait(&bar.x_full, 0, a.err);
      // S and dP of a tile: stage st, its phase, group g.
      auto scores = [&](int st, int par, int g) {
        ok = warp_wait(&bar.full[st], par, a.err) && !*dead;
        if (!ok) return;
        tc_fence_after();
        const uint64_t ud = u_desc + (uint32_t)st * (S::kStage >> 4);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int s = 0; s < DP / 16; ++s)
            if (s < ksteps)
              mma_ss(leader, tmem + g * 128 + 64 * y,
                     x_desc + ((y * S::kX + (s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4),
                     ud + ((y * S::kTile + (s >> 2) * (kTileRows * 128) + (s & 3) * 32) >> 4),
                     kShapeS, s > 0);
        mma_commit(leader, &bar.s_full[g]);
      };
      int lst = 0, lpar = 0, lg = 0;  // of the next tile to score
      auto advance = [&](int& st, int& par, int& g) {
        if (++st == S::kStages) st = 0, par ^= 1;
        if (++g == G) g = 0;
      };
      for (int t = 0; ok && t < G && t < total; ++t) {
        scores(lst, lpar, lg);
        advance(lst, lpar, lg);
      }
      int st = 0, par = 0, g = 0, gpar = 0;
      for (int t = 0; ok && t < total; ++t) {
        ok = warp_wait(&bar.p_full[g], gpar, a.err) && !*dead;
        if (!ok) break;
        tc_fence_after();
        const uint64_t ud = u_rows + (uint32_t)st * (S::kStage >> 4);
        if (!DQ) {
#pragma unroll
          for (int s = 0; s < kTileRows / 16; ++s)
            mma_ts(leader, tmem + S::kAcc, tmem + g * 128 + s * 8,
                   ud + ((S::kTile + s * 2048) >> 4), kShapeA, t > 0 || s > 0);
        }
#pragma unroll
        for (int s = 0; s < kTileRows / 16; ++s)
          mma_ts(leader, tmem + S::kAcc + (DQ ? 0 : DP), tmem + g * 128 + 64 + s * 8,
                 ud + (s * 2048 >> 4), kShapeA, t > 0 || s > 0);
        // Only where a later copy waits for it: nothing may arrive after the block's end.
        if (t + S::kStages < total) mma_commit(leader, &bar.empty[st]);
        if (t + G < total) {
          scores(lst, lpar, lg);
          advance(lst, lpar, lg);
        }
        advance(st, par, g);
        if (g == 0) gpar ^= 1;
      }
      if (!ok) *dead = 1;
      mma_commit(leader, &bar.done);
      if (!ok) mbar_wait(&bar.done, 0, a.err, kErrDrain);
    }
  } else {
    // ----- arithmetic: a thread a row of X ----------------------------------
    const int g = warp >> 2, row = (warp & 3) * 32 + lane, x = x0 + row;
    const int wx = x0 + (warp & 3) * 32;  // the warp's first row
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + g * 128, tp = ts + 64;
    const uint64_t per_row = (uint32_t)((a.Lk + 7) / 8);
    float nlse = 0.0f, ndelta = 0.0f;  // of the row's query
    if (DQ) {  // Lqp covers every row of the block
      const float* r = a.rows + row_at(b * a.H + h0, a.Lqp, x);
      nlse = r[0];
      ndelta = r[kTileRows];
    }
    const uint32_t T2 = a.keep.T * 0x10001u;
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
    float far_left = 0.0f, far_right = 0.0f;
    bool ok = true;
    int t = g;  // this group's next tile
    for (int hh = 0; hh < heads; ++hh) {
      const int h = h0 + hh;
      if (a.biased) {
        if (!DQ) {  // the head's bias; every group passes here once a head
          named_sync(1, 128 * G);
          stage_bias(bias, a.rp, bar.first, static_cast<const T*>(a.table), a.H, h, threadIdx.x,
                     128 * G);
          named_sync(1, 128 * G);
        }
        far_left = bias[0];
        far_right = bias[nbias - 1];
      }
      const uint64_t rows0 = (uint64_t)(b * a.H + h) * a.Lq;
      for (; ok && t < (hh + 1) * per; t += G) {
        const int st = t % S::kStages;
        const int c0 = (from + t - hh * per) * kTileRows;  // first column (key or query)
        uint8_t* stage = smem + 2 * S::kX + st * S::kStage;
        // The keep bits do not wait for the scores.
        uint32_t kept[2] = {~0u, ~0u};
        if (!DQ && DROP) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            kept[u] = keep_column(
                a.keep,
                (rows0 + (uint32_t)(c0 + 32 * u + (lane & 7))) * per_row + (uint32_t)(x >> 3),
                per_row, lane);
        }
        ok = warp_wait(&bar.s_full[g], (t / G) & 1, a.err);
        if (!ok) break;
        tc_fence_after();
        uint32_t rs[2][16], rp[2][16];
        tmem_ld16(rs[0], ts);
        tmem_ld16(rp[0], tp);
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // 32 columns at a time
          const int col = c0 + 32 * u;
          // distance of the warp's first row and the first column
          const int d = DQ ? col - wx - a.q_offset : wx - col - a.q_offset;
          bool near = false;
          float far = 0.0f;
          if (a.biased) {
            near = d + 31 > -span.left && d - 31 < span.right;
            far = d > 0 ? far_right : far_left;
          }
          const bool masked = DQ ? col + 32 > warp_limit : col < warp_limit;
          const float* tb = bias + (DQ ? col - x : x - col) - a.q_offset + span.left + kBiasMargin;
          float ds[32];
          uint64_t mass = 0;  // sums of p, two lanes of them
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int cc = 2 * u + hf;  // 16 columns; the next 16 are on their way meanwhile
            tmem_wait_ld(rs[cc & 1]);
            tmem_wait_ld(rp[cc & 1]);
            if (cc < 3) {
              tmem_ld16(rs[~cc & 1], ts + 16 * (cc + 1));
              tmem_ld16(rp[~cc & 1], tp + 16 * (cc + 1));
            }
            const uint32_t(&vs)[16] = rs[cc & 1];
            const uint32_t(&vp)[16] = rp[cc & 1];
            const uint64_t scale2 = pair(a.scale2, a.scale2);
            const ulonglong2* qlse =  // two pairs of queries each
                reinterpret_cast<const ulonglong2*>(stage + 2 * S::kTile) + 4 * cc;
            const ulonglong2* qdelta = qlse + kTileRows / 4;
            float p[16];
            auto score = [&](int k, uint64_t shift) {
              unpair(fma2(pair(vs[2 * k], vs[2 * k + 1]), scale2, shift), &p[2 * k], &p[2 * k + 1]);
            };
            if (near) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int n = 16 * hf + 2 * k;
                const uint64_t bias2 = DQ ? pair(tb[n], tb[n + 1]) : pair(tb[-n], tb[-n - 1]);
                if (DQ) {
                  score(k, add2(bias2, pair(nlse, nlse)));
                } else {
                  const ulonglong2 four = qlse[k >> 1];
                  score(k, add2(bias2, k & 1 ? four.y : four.x));
                }
              }
            } else if (DQ) {
              const float f = far + nlse;
#pragma unroll
              for (int k = 0; k < 8; ++k) score(k, pair(f, f));
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const ulonglong2 four = qlse[k >> 1];
                score(k, add2(pair(far, far), k & 1 ? four.y : four.x));
              }
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) p[k] = exp2_approx(p[k]);
            if (masked) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                p[k] = (DQ ? col + 16 * hf + k < limit : col + 16 * hf + k >= limit) ? p[k] : 0.0f;
            }
            float z[16];
            if (DROP && DQ) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint4 w = keep_words(a.keep, (rows0 + (uint32_t)x) * per_row +
                                                       (uint32_t)((col >> 3) + 2 * hf + k));
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  keep_pair(v[e], T2, p[8 * k + 2 * e], p[8 * k + 2 * e + 1],
                            &z[8 * k + 2 * e], &z[8 * k + 2 * e + 1]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                z[k] = !DROP || (kept[u] >> (16 * hf + k) & 1) ? p[k] : 0.0f;
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
              unpair(fma2(pair(z[2 * k], z[2 * k + 1]), pair(vp[2 * k], vp[2 * k + 1]), mul2(pp, nd)),
                     &ds[16 * hf + 2 * k], &ds[16 * hf + 2 * k + 1]);
              if (DQ) mass = add2(mass, pp);
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                float& e = ds[16 * hf + k];
                e = (DQ ? col + 16 * hf + k < limit : col + 16 * hf + k >= limit) ? e : 0.0f;
              }
            }
            uint32_t o[8];
            if (!DQ) {
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = pack2<T>(z[2 * k], z[2 * k + 1]);
              tmem_st8(ts + 8 * cc, o);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o[k] = pack2<T>(ds[16 * hf + 2 * k], ds[16 * hf + 2 * k + 1]);
            tmem_st8(tp + 8 * cc, o);
          }
          if (sums) {
            uint64_t s2 = 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) s2 = add2(s2, pair(ds[2 * k], ds[2 * k + 1]));
            float s0, s1;
            unpair(s2, &s0, &s1);
            const float sum = s0 + s1;
            eps += sum;
            if (!near) {
              unpair(mass, &s0, &s1);
              if (d > 0) {
                far_r += sum;
                mass_r += s0 + s1;
              } else {
                far_l += sum;
                mass_l += s0 + s1;
              }
            } else {
              // Sums down the diagonals of the 32 x 32 block: a running sum moves one
              // lane (row) on with every column; what lane 31 holds is complete.
              float run = 0.0f;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float up = __shfl_up_sync(0xffffffffu, run, 1);
                run = lane ? up + ds[k] : ds[k];
                if (lane == 31) bar.carry[warp][k] = run;
              }
              __syncwarp();
              float* to = by_d + warp * nbias + d + span.left + kBiasMargin;
              if (lane < 31) to[lane - 31] += bar.carry[warp][lane];
              __syncwarp();
              to[31 - lane] += run;
              __syncwarp();
            }
          }
        }
        tmem_wait_st();
        if (DQ && keys < a.Lk && c0 + kTileRows > keys) {
          // Rows of K past the length have dS = 0, but may hold anything.
          const int live = keys - c0;
          for (int k = threadIdx.x & 127; k < (kTileRows - live) * 8 * (DP / 64); k += 128) {
            const int r = live + (k >> 3) % (kTileRows - live), y = (k >> 3) / (kTileRows - live);
            *reinterpret_cast<uint4*>(stage + y * (kTileRows * 128) + r * 128 + (k & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        tc_fence_before();
        mbar_arrive(&bar.p_full[g]);
      }
    }
    if (ok && total > 0) ok = warp_wait(&bar.done, 0, a.err);
    if (!ok) *dead = 1;
    tc_fence_after();

    // ----- results --------------------------------------------------------------
    const int rows_x = DQ ? a.Lq : a.Lk;
    const bool none = total == 0 || (!DQ && x >= keys);
#pragma unroll 1
    for (int c = g; c < (DQ ? 1 : 2) * DP / 32; c += G) {
      uint32_t r[32];
      if (total > 0) {
        tmem_ld32(r, tmem + lanes + S::kAcc + 32 * c);
        tmem_wait_ld(r);
      }
      const bool second = DQ || c >= DP / 32;
      const Heads& out = second ? a.out2 : a.out1;
      const int col = 32 * (DQ ? c : c % (DP / 32));
      const float mul = second ? a.scale * a.keep.scale : a.keep.scale;
      T* to = static_cast<T*>(out.data) + b * out.b + (int64_t)x * out.l + hx * out.h + col;
      if (x < rows_x) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (col + 8 * k >= a.D) break;
          uint32_t o[4] = {0, 0, 0, 0};
          if (!none) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack2<T>(__uint_as_float(r[8 * k + 2 * e]) * mul,
                              __uint_as_float(r[8 * k + 2 * e + 1]) * mul);
          }
          *reinterpret_cast<uint4*>(to + 8 * k) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    if (sums) {
      // A row's dS sums to zero; what it sums to is the error of rowsum(do o),
      // taken from the rounded o.  It is taken out of the far buckets, whose
      // weight would multiply it, and out of the row's entry for dk.
      bar.eps[g][row] = eps;
      named_sync(1, 128 * G);
      float e = 0.0f;
#pragma unroll
      for (int k = 0; k < G; ++k) e += bar.eps[k][row];
      if (g == 0)
        a.rows[row_at(b * a.H + h0, a.Lqp, x) + kTileRows] = ndelta - e;
      far_l -= e * mass_l;
      far_r -= e * mass_r;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        far_l += __shfl_xor_sync(0xffffffffu, far_l, o);
        far_r += __shfl_xor_sync(0xffffffffu, far_r, o);
      }
      if (lane == 0) {
        bar.far[warp][0] = far_l;
        bar.far[warp][1] = far_r;
      }
      named_sync(1, 128 * G);
      const int last_l = a.rp.side - 1, last_r = a.rp.two_sided ? a.rp.num_buckets - 1 : 0;
      float* to = a.partial + (((int64_t)h0 * a.B + b) * gridDim.x + blockIdx.x) * a.rp.num_buckets;
      for (int k = warp; k < a.rp.num_buckets; k += S::kWarps) {
        int64_t lo, hi;
        bucket_range(bar.first, a.rp.side, a.rp.two_sided, k, -(span.left + kBiasMargin),
                     span.right + kBiasMargin, &lo, &hi);
        float sum = 0.0f;
        for (int i = (int)lo + span.left + kBiasMargin + lane;
             i < (int)hi + span.left + kBiasMargin; i += 32)
#pragma unroll
          for (int w = 0; w < S::kWarps; ++w) sum += by_d[w * nbias + i];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
          for (int w = 0; w < S::kWarps; ++w) {
            if (k == last_l) sum += bar.far[w][0];
            if (k == last_r) sum += bar.far[w][1];
          }
          to[k] = sum * a.keep.scale;
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == kProducts) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <typename T, int DP, bool DQ, bool DROP>
cudaError_t grad_of(const AttnArgs& a, GradArgs f, cudaStream_t s) {
  using S = GradShape<DP, DQ>;
  // An empty side is never read; its map still needs an address and an extent.
  auto map = [&](CUtensorMap* m, const Heads& t, int L, int heads, int rows) {
    return L ? attn_tensor_map(m, t, a.type, a.D, L, heads, a.B, rows)
             : attn_tensor_map(m, DQ ? a.q : a.k, a.type, a.D, 1, 1, 1, rows);
  };
  const int Lx = DQ ? a.Lq : a.Lk, Lu = DQ ? a.Lk : a.Lq;
  const int Hx = DQ ? a.H : a.Hkv, Hu = DQ ? a.Hkv : a.H;
  cudaError_t e = map(&f.x, DQ ? a.q : a.k, Lx, Hx, kRows);
  if (e == cudaSuccess) e = map(&f.y, DQ ? a.grad_o : a.v, Lx, Hx, kRows);
  if (e == cudaSuccess) e = map(&f.u, DQ ? a.k : a.q, Lu, Hu, kTileRows);
  if (e == cudaSuccess) e = map(&f.w, DQ ? a.v : a.grad_o, Lu, Hu, kTileRows);
  if (e != cudaSuccess) return e;
  f.out1 = DQ ? a.dq : a.dv;
  f.out2 = DQ ? a.dq : a.dk;
  constexpr size_t most = 1024 + S::kBias + kBiasMostBytes * (DQ ? 1 + S::kWarps : 1);
  const size_t bytes = 1024 + S::kBias +
                       (a.biased ? bias_floats(a.rp) * 4 * (f.partial ? 1 + S::kWarps : 1) : 0);
  static PerDeviceOnce once;
  e = once.run([] {
    return cudaFuncSetAttribute(k_attn_grad<T, DP, DQ, DROP>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((Lx + kRows - 1) / kRows, a.B * Hx);
  k_attn_grad<T, DP, DQ, DROP><<<grid, S::kThreads, bytes, s>>>(f);
  return cudaGetLastError();
}

template <typename T, bool DQ>
cudaError_t grad(const AttnArgs& a, const GradArgs& f, cudaStream_t s) {
  if (a.D <= 64)
    return a.keep.T ? grad_of<T, 64, DQ, true>(a, f, s) : grad_of<T, 64, DQ, false>(a, f, s);
  return a.keep.T ? grad_of<T, 128, DQ, true>(a, f, s) : grad_of<T, 128, DQ, false>(a, f, s);
}

int padded(int Lq) { return (Lq + kRows - 1) / kRows * kRows; }

size_t rows_bytes(const AttnArgs& a) {
  return ((size_t)a.B * a.H * padded(a.Lq) * 2 * sizeof(float) + 255) / 256 * 256;
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
  f.rows = static_cast<float*>(a.workspace);
  f.Lqp = padded(a.Lq);
  if (a.Lq) {
    RowArgs r{a.B, a.H, a.D, a.Lq, f.Lqp, a.o, a.grad_o, a.lse, 1.0f / a.keep.scale, f.rows};
    const int64_t rows = (int64_t)a.B * a.H * f.Lqp;
    k_rows<T><<<(unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock), 16 * kRowsPerBlock, 0, s>>>(r);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.dtable) f.partial = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + rows_bytes(a));
    e = grad<T, true>(a, f, s);
    if (e != cudaSuccess) return e;
    if (a.dtable) {
      e = launch_bucket_sums(f.partial, a.B * ((a.Lq + kRows - 1) / kRows), a.H, a.rp.num_buckets,
                             a.dtable, a.type, s);
      if (e != cudaSuccess) return e;
      f.partial = nullptr;
    }
  }
  if (a.Lk) e = grad<T, false>(a, f, s);
  return e;
}

}  // namespace

size_t attn_workspace_bytes(const AttnArgs& a) {
  size_t n = rows_bytes(a);
  if (a.biased)
    n += (size_t)a.B * a.H * ((a.Lq + kRows - 1) / kRows) * a.rp.num_buckets * sizeof(float);
  return n;
}

cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s) {
  if (a.dtable && (a.B == 0 || a.Lq == 0)) {
    const cudaError_t e = cudaMemsetAsync(a.dtable, 0, (size_t)a.rp.num_buckets * a.H * 2, s);
    if (e != cudaSuccess) return e;
  }
  if (a.B == 0) return cudaSuccess;
  return a.type == OB_TYPE_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<__half>(a, s);
}

}  // namespace ob
