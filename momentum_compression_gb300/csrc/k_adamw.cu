// AdamW over many tensors, one launch for up to 512 of them.
//
// A warp takes blocks of 256 elements, eight of each a lane.  The table of
// tensors comes as the kernel's parameter: pointers may change from call to
// call, nothing is copied, and a graph keeps what it captured.
//
// Moments in 8 bits: a block's largest value gives its unit, a power of two, so
// that scaling is exact; a code is the value's bits in that unit, plus 16 random
// bits, cut off after three bits of significand.  The random bits are what lets
// v fall: 0.1% a step is far below half a code.
#include <cmath>

#include "elem.cuh"
#include "layers.cuh"
#include "philox.cuh"

namespace ob {
namespace {

constexpr int kAdamThreads = 256;

template <int CAP>
struct AdamTable {
  AdamTensor t[CAP];
};

struct AdamCall {
  AdamArgs a;
  PhiloxKeys keys;
  uint64_t first, blocks;  // of the state, in this launch
  int count, last;         // last: this launch advances the counter
  float b1, c1, b2, c2;    // c = 1 - b
};

struct AdamStep {  // of the whole call
  float lr, size, root, scale;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), the gradients' factor
  uint32_t lo, hi;              // t
  int skip;
};

// Codes of a moment: an exponent field with bias BIAS, three bits of significand.
template <int BIAS>
__device__ __forceinline__ float decode(uint32_t c, float unit) {
  constexpr uint32_t nan = BIAS == 7 ? 127u : 255u;
  const uint32_t size = BIAS == 7 ? c & 127u : c;
  // as fp32 bits it is the value times 2^(BIAS - 127), below the normal range too
  const float v = __uint_as_float(size << 20) * __uint_as_float((uint32_t)(254 - BIAS) << 23) * unit;
  if (size == nan) return __uint_as_float(0x7fffffffu);
  return BIAS == 7 && (c & 128u) ? -v : v;
}
__device__ __forceinline__ float unit_of(uint32_t e) { return __uint_as_float(e << 23); }

// E of a block whose largest finite value has bits `top`.
template <int BIAS>
__device__ __forceinline__ int block_exp(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  return top == 0 ? 0 : min(max(e, BIAS == 7 ? 1 : 3), 246);
}

template <int BIAS>
__device__ __forceinline__ uint32_t encode(float x, float up, uint32_t noise) {
  constexpr int most = BIAS == 7 ? 126 : 254;
  const float size = fabsf(x), y = size * up;
  int c = (int)((__float_as_uint(y) + (noise << 4)) >> 20) - ((127 - BIAS) << 3);
  const int low = (int)((uint32_t)__float2int_rz(y * (float)(1ull << (18 + BIAS))) + noise) >> 16;
  if (y < __uint_as_float((uint32_t)(128 - BIAS) << 23)) c = low;
  c = min(c, most);
  if (BIAS != 7 && size > 0.0f) c = max(c, 1);
  if (!(size < INFINITY)) c = most + 1;
  return (uint32_t)c | (BIAS == 7 ? __float_as_uint(x) >> 24 & 128u : 0u);
}

template <int CAP, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads)
    k_adamw(const __grid_constant__ AdamCall c, const __grid_constant__ AdamTable<CAP> table) {
  __shared__ AdamStep shared_step;
  const AdamArgs& a = c.a;
  if (threadIdx.x == 0) {
    AdamStep s;
    const double t = a.counter[0] + 1.0, b1t = a.counter[1] * a.b1, b2t = a.counter[2] * a.b2;
    s.lr = a.lr_device ? *a.lr_device : (float)a.lr;
    s.size = (float)((a.lr_device ? (double)s.lr : a.lr) / (1.0 - b1t));
    s.root = (float)(1.0 / sqrt(1.0 - b2t));
    s.scale = a.grad_scale ? *a.grad_scale : 1.0f;
    const uint64_t n = (uint64_t)t;
    s.lo = (uint32_t)n;
    s.hi = (uint32_t)(n >> 32);
    s.skip = a.skip && *a.skip != 0.0f;
    shared_step = s;
  }
  __syncthreads();
  const AdamStep s = shared_step;
  const int lane = threadIdx.x & 31;
  const uint64_t warp = (uint64_t)blockIdx.x * (kAdamThreads / 32) + (threadIdx.x >> 5);
  const uint64_t warps = (uint64_t)gridDim.x * (kAdamThreads / 32);
  if (!s.skip)
    for (uint64_t i = warp; i < c.blocks; i += warps) {
      const uint64_t b = c.first + i;
      int lo = 0, hi = c.count;  // table.t[lo].first <= b < table.t[hi].first
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.t[mid].first <= b)
          lo = mid;
        else
          hi = mid;
      }
      const AdamTensor& t = table.t[lo];
      if (!t.g) continue;
      const uint64_t at = (b - t.first) * kAdamBlock + lane * 8;  // in the tensor
      const uint64_t st = b * kAdamBlock + lane * 8;              // in the state
      const int n = at < t.n ? (int)min((uint64_t)8, t.n - at) : 0;
      float m[8], v[8];
      if constexpr (EIGHT) {
        const uint2 mc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + st);
        const uint2 vc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + st);
        const float um = unit_of(a.m_exp[b]), uv = unit_of(a.v_exp[b]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = decode<7>((k < 4 ? mc.x : mc.y) >> (8 * (k & 3)) & 255u, um);
          v[k] = decode<23>((k < 4 ? vc.x : vc.y) >> (8 * (k & 3)) & 255u, uv);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m[k] = static_cast<float*>(a.m)[st + k];
          v[k] = static_cast<float*>(a.v)[st + k];
        }
      }
      const float keep = 1.0f - s.lr * t.decay;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (k >= n) {
          m[k] = v[k] = 0.0f;
          continue;
        }
        const float g = load_as_f32(t.g, at + k, a.g_type) * s.scale;
        m[k] = __fadd_rn(__fmul_rn(m[k], c.b1), __fmul_rn(g, c.c1));
        v[k] = __fadd_rn(__fmul_rn(v[k], c.b2), __fmul_rn(__fmul_rn(g, c.c2), g));
        const float p = load_as_f32(t.p, at + k, t.types & 255);
        const float den = __fmaf_rn(sqrtf(v[k]), s.root, a.eps);
        const float q = __fmaf_rn(-s.size, m[k] / den, p * keep);
        store_from_f32(t.p, at + k, t.types & 255, q);
        if (t.copy) store_from_f32(t.copy, at + k, t.types >> 8, q);
      }
      if constexpr (EIGHT) {
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t x = __float_as_uint(m[k]) & 0x7fffffffu, y = __float_as_uint(v[k]);
          if (x < 0x7f800000u) tm = max(tm, x);
          if (y < 0x7f800000u) tv = max(tv, y);
        }
        const int em = block_exp<7>(__reduce_max_sync(0xffffffffu, tm));
        const int ev = block_exp<23>(__reduce_max_sync(0xffffffffu, tv));
        const float upm = em ? __uint_as_float((uint32_t)(254 - em) << 23) : 0.0f;
        const float upv = ev ? __uint_as_float((uint32_t)(254 - ev) << 23) : 0.0f;
        uint32_t mo[2] = {0, 0}, vo[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t call = st / 4 + h;
          const uint4 w = philox4x32_10(
              make_uint4((uint32_t)call, (uint32_t)(call >> 32), s.lo, s.hi), c.keys);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t r = word_of(w, k);
            mo[h] |= encode<7>(m[4 * h + k], upm, r & 0xffffu) << (8 * k);
            vo[h] |= encode<23>(v[4 * h + k], upv, r >> 16) << (8 * k);
          }
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + st) = make_uint2(mo[0], mo[1]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + st) = make_uint2(vo[0], vo[1]);
        if (lane == 0) {
          a.m_exp[b] = (uint8_t)em;
          a.v_exp[b] = (uint8_t)ev;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          static_cast<float*>(a.m)[st + k] = m[k];
          static_cast<float*>(a.v)[st + k] = v[k];
        }
      }
    }
  // The block that ends last has seen all others read the counter.
  if (!c.last || s.skip) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* ticket = reinterpret_cast<unsigned*>(a.counter + 3);
    if (atomicAdd(ticket, 1u) == gridDim.x - 1) {
      *ticket = 0;
      a.counter[0] += 1.0;
      a.counter[1] *= a.b1;
      a.counter[2] *= a.b2;
    }
  }
}

// The moments' values, which bf16 holds exactly (but below 2^-126).
__global__ void __launch_bounds__(256)
    k_moments(const uint8_t* m, const uint8_t* v, const uint8_t* m_exp, const uint8_t* v_exp,
              uint64_t blocks, uint32_t* m_out, uint32_t* v_out) {
  const int lane = threadIdx.x & 31;
  const uint64_t b = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (b >= blocks) return;
  const uint64_t st = b * kAdamBlock + lane * 8;
  auto one = [&](const uint8_t* codes, const uint8_t* exps, uint32_t* out, auto bias) {
    const uint2 c = *reinterpret_cast<const uint2*>(codes + st);
    const float u = unit_of(exps[b]);
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      x[k] = decode<decltype(bias)::value>((k < 4 ? c.x : c.y) >> (8 * (k & 3)) & 255u, u);
    using B = __nv_bfloat16;
    *reinterpret_cast<uint4*>(out + st / 2) = make_uint4(
        pack2<B>(x[0], x[1]), pack2<B>(x[2], x[3]), pack2<B>(x[4], x[5]), pack2<B>(x[6], x[7]));
  };
  one(m, m_exp, m_out, std::integral_constant<int, 7>());
  one(v, v_exp, v_out, std::integral_constant<int, 23>());
}

template <int CAP>
cudaError_t launch(const AdamCall& c, const AdamTensor* t, cudaStream_t s) {
  AdamTable<CAP> table;
  for (int i = 0; i < c.count; ++i) table.t[i] = t[i];
  const uint64_t want = (c.blocks + kAdamThreads / 32 - 1) / (kAdamThreads / 32);
  const int grid = (int)(want < 1 ? 1 : want < 1216 ? want : 1216);
  if (c.a.bits == 8)
    k_adamw<CAP, true><<<grid, kAdamThreads, 0, s>>>(c, table);
  else
    k_adamw<CAP, false><<<grid, kAdamThreads, 0, s>>>(c, table);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamArgs& a, const AdamTensor* t, int count, cudaStream_t s) {
  constexpr int kMost = 512;
  AdamCall c{};
  c.a = a;
  c.keys = philox_keys((uint32_t)a.seed, (uint32_t)(a.seed >> 32));
  c.b1 = (float)a.b1;
  c.c1 = (float)(1.0 - a.b1);
  c.b2 = (float)a.b2;
  c.c2 = (float)(1.0 - a.b2);
  int at = 0;
  do {
    c.count = count - at < kMost ? count - at : kMost;
    c.last = at + c.count == count;
    c.first = c.count ? t[at].first : 0;
    c.blocks = 0;
    if (c.count) {
      const AdamTensor& end = t[at + c.count - 1];
      c.blocks = end.first + (end.n + kAdamBlock - 1) / kAdamBlock - c.first;
    }
    cudaError_t e = c.count <= 16    ? launch<16>(c, t + at, s)
                    : c.count <= 128 ? launch<128>(c, t + at, s)
                                     : launch<kMost>(c, t + at, s);
    if (e != cudaSuccess) return e;
    at += c.count;
  } while (at < count);
  return cudaSuccess;
}

cudaError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const uint8_t* m_exp,
                                 const uint8_t* v_exp, size_t elements, void* m_out, void* v_out,
                                 cudaStream_t s) {
  const uint64_t blocks = elements / kAdamBlock;
  if (blocks)
    k_moments<<<(unsigned)((blocks + 7) / 8), 256, 0, s>>>(
        m, v, m_exp, v_exp, blocks, static_cast<uint32_t*>(m_out), static_cast<uint32_t*>(v_out));
  return cudaGetLastError();
}

}  // namespace ob
