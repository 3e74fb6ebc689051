// What the attention's forward and backward kernels share: the argument
// block, the tensor maps of its arrays, the staged bias, the keep bits.
#pragma once

#include <cuda.h>

#include "elem.cuh"
#include "model.cuh"

namespace ob {

// Element (b, i, h, d) at data + b * this->b + i * l + h * this->h + d.
struct Heads {
  void* data;
  int64_t b, l, h;
};

struct AttnArgs {
  int type, B, H, Hkv, D, Lq, Lk, causal, q_offset, biased;
  float scale;
  ob_relpos rp;
  const void* table;
  const int32_t* kv_len;
  Keep keep;
  Heads q, k, v, o, grad_o, dq, dk, dv;
  float* lse;  // [B][H][Lq], or null
  void* dtable;
  void* workspace;
};

size_t attn_workspace_bytes(const AttnArgs& a);
cudaError_t launch_attn_fwd(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_bwd(const AttnArgs& a, cudaStream_t s);

// The device word where a wait that ran out leaves its code.
cudaError_t attn_error_word(unsigned** word);

// A map of one array whose boxes are `rows` rows of 64 elements of one head:
// elements past D and rows past L read as zero.
cudaError_t attn_tensor_map(CUtensorMap* map, const Heads& t, int type, int D, int L, int H, int B,
                            int rows);

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

#ifdef __CUDACC__

// Keys of batch entry b that any query sees.  The others may hold anything: what
// comes after them in a tile is masked, and cleared where a zero weight meets it.
template <typename Args>
__device__ __forceinline__ int key_count(const Args& a, int b) {
  int n = a.kv_len ? min(a.Lk, a.kv_len[b]) : a.Lk;
  if (a.causal) n = min(n, a.Lq + a.q_offset);
  return max(0, n);
}

// ---------------------------------------------------------------------------
// Bias.  Distances up to -left share one bucket and so do those from right on;
// between them (and kBiasMargin past either end, so that a block of 32 x 64
// that touches the range is covered whole) the values of one head, times
// log2(e), are staged in shared memory.
// ---------------------------------------------------------------------------

constexpr int kBiasMargin = 96;
constexpr int kBiasMost = OB_ATTN_MAX_SPAN + 2 * kBiasMargin + 1;  // floats
constexpr int kBiasMostBytes = 4 * kBiasMost;

struct BiasSpan {
  int left, right;
};
__host__ __device__ inline BiasSpan bias_span(const ob_relpos& rp) {
  const int last = rp.first[rp.side - 1];
  return BiasSpan{last, rp.two_sided ? last : 0};
}
__host__ __device__ inline int bias_floats(const ob_relpos& rp) {
  const BiasSpan s = bias_span(rp);
  return s.left + s.right + 2 * kBiasMargin + 1;
}

// Buckets of the staged distances (entry t: distance t - left - margin), by
// threads tid of n; rp is the kernel's parameter.
__device__ __forceinline__ void stage_buckets(uint8_t* map, const ob_relpos& rp, int tid, int n) {
  const BiasSpan s = bias_span(rp);
  const int count = s.left + s.right + 2 * kBiasMargin + 1;
  for (int t = tid; t < count; t += n)
    map[t] = (uint8_t)bucket_of(rp.first, rp.side, rp.two_sided, t - s.left - kBiasMargin);
}
// Finite values count up to 2^16 either way.  bf16's extremes times log2(e) would
// be infinite, and a row whose keys all have one has to come out as if it had
// none: the difference of such a value and the row's lse, both rounded near
// 2^16, is off by 1% of a weight, and by all of it from 2^23 on.  -inf masks.
constexpr float kBiasLimit = 65536.0f;
template <typename T>
__device__ __forceinline__ void stage_bias(float* tab, const uint8_t* map, int count,
                                           const T* table, int H, int h, int tid, int n) {
#pragma unroll 8
  for (int t = tid; t < count; t += n) {
    const float x = to_f32(table[(size_t)map[t] * H + h]);
    const float size = fabsf(x);
    tab[t] = (size > kBiasLimit && size < INFINITY ? copysignf(kBiasLimit, x) : x) * kLog2e;
  }
}

// ---------------------------------------------------------------------------
// Keep bits, eight a call: a word's two as masks of 16 bits.  Non-negative
// bf16 patterns are ordered like whole numbers, so u < T is one compare of the
// packed 16-bit pipe for both; the NaN patterns, above every number, count as
// kept (geu), and T is at most infinity's, 0x7f80.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t keep_mask2(uint32_t w, uint32_t T2) {
  uint32_t m;
  asm("{\n\t.reg .b32 u;\n\tabs.bf16x2 u, %1;\n\tset.geu.u32.bf16x2 %0, u, %2;\n\t}"
      : "=r"(m)
      : "r"(w), "r"(T2));
  return m;
}

#endif

}  // namespace ob
