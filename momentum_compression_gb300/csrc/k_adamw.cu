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
constexpr int kAdamGrid = 3 * 152;  // all that run at a time

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

// ---------------------------------------------------------------------------
// Moments in 8 bits
// ---------------------------------------------------------------------------

__device__ __forceinline__ float power_of_two(int e) {  // biased, 1..254
  return __uint_as_float((uint32_t)e << 23);
}

// Four codes of m, which are floats of a type that the hardware converts.
__device__ __forceinline__ void decode_m(uint32_t w, float unit, float* m) {
  uint32_t h[2];
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 f = unpack2<__half>(h[k]);
    m[2 * k] = f.x * unit;
    m[2 * k + 1] = f.y * unit;
  }
}
// Four of v: as fp32 bits, twenty places up, a code is its value times 2^-104, below the
// normal range too.  `up` is 2^104 times the unit as far as fp32 goes, `more` the rest.
struct VUnit {
  float up, more;
  __device__ __forceinline__ explicit VUnit(int e) {
    up = e ? power_of_two(min(e + 104, 254)) : 0.0f;
    more = power_of_two(max(e + 104 - 254, 0) + 127);
  }
};
__device__ __forceinline__ void decode_v(uint32_t w, const VUnit& u, float* v) {
  v[0] = __uint_as_float((w << 20) & 0x0ff00000u) * u.up;
  v[1] = __uint_as_float((w << 12) & 0x0ff00000u) * u.up;
  v[2] = __uint_as_float((w << 4) & 0x0ff00000u) * u.up;
  v[3] = __uint_as_float((w >> 4) & 0x0ff00000u) * u.up;
  if (u.more != 1.0f)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= u.more;
  if (__vcmpeq4(w, 0xffffffffu))
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((w >> (8 * k) & 255u) == 255u) v[k] = __uint_as_float(0x7fffffffu);
}

// E of a block whose largest finite value has bits `top`.
template <int BIAS>
__device__ __forceinline__ int block_exp(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  return top == 0 ? 0 : min(max(e, BIAS == 7 ? 1 : 3), 246);
}

// The code of size >= 0, finite, in the unit 1 / up, `noise` the random bits four places
// up: below the normal codes the smallest normal one is added first, toward zero, which
// makes the same steps of the float's bits.  No value of a block passes the largest
// code, whose unit goes by them all.
template <int BIAS>
__device__ __forceinline__ uint32_t encode(float size, float up, uint32_t noise) {
  constexpr uint32_t kBase = (uint32_t)(127 - BIAS) << 23;  // bits of half the smallest normal code
  const float y = size * up, least = __uint_as_float(kBase + (1u << 23));
  const uint32_t bits =
      y < least ? __float_as_uint(__fadd_rz(y, least)) - (1u << 23) : __float_as_uint(y);
  uint32_t c = (bits + noise - kBase) >> 20;
  if (BIAS != 7) c = max(c, min(__float_as_uint(size), 1u));
  return c;
}
// The same for any x: what is not finite has the code after the last.
template <int BIAS>
__device__ __forceinline__ uint32_t encode_any(float size, float up, uint32_t noise) {
  constexpr uint32_t most = BIAS == 7 ? 126 : 254;
  return size < INFINITY ? min(encode<BIAS>(size, up, noise), most) : most + 1;
}

// ---------------------------------------------------------------------------
// Eight elements of a lane
// ---------------------------------------------------------------------------

__device__ __forceinline__ void load_f32x8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void store_f32x8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack2<T>(w[k]);
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                    pack2<T>(v[6], v[7]));
}

// n of the eight from element `at` of p; whole: all eight, aligned.
__device__ __forceinline__ void load8(const void* p, uint64_t at, int type, bool whole, int n,
                                      float (&v)[8]) {
  if (!whole) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? load_as_f32(p, at + k, type) : 0.0f;
  } else if (type == OB_TYPE_F32) {
    load_f32x8(static_cast<const float*>(p) + at, v);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    if (type == OB_TYPE_BF16)
      unpack8<__nv_bfloat16>(u, v);
    else
      unpack8<__half>(u, v);
  }
}
__device__ __forceinline__ void store8(void* p, uint64_t at, int type, bool whole, int n,
                                       const float (&v)[8]) {
  if (!whole) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store_from_f32(p, at + k, type, v[k]);
  } else if (type == OB_TYPE_F32) {
    store_f32x8(static_cast<float*>(p) + at, v);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        type == OB_TYPE_BF16 ? pack8<__nv_bfloat16>(v) : pack8<__half>(v);
  }
}

__device__ __forceinline__ float sqrt_near(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int CAP, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads, 3)
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
      const uint64_t begin = (b - t.first) * kAdamBlock, at = begin + lane * 8;  // in the tensor
      const uint64_t st = b * kAdamBlock + lane * 8;                             // in the state
      const int n = at < t.n ? (int)min((uint64_t)8, t.n - at) : 0;
      const bool full = begin + kAdamBlock <= t.n;
      const bool whole = full && (t.types >> 16);
      const int p_type = t.types & 255, copy_type = t.types >> 8 & 255;
      float g[8], p[8], m[8], v[8];
      load8(t.g, at, a.g_type, whole, n, g);
      load8(t.p, at, p_type, whole, n, p);
      if constexpr (EIGHT) {
        const uint2 mc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.m) + st);
        const uint2 vc = *reinterpret_cast<const uint2*>(static_cast<uint8_t*>(a.v) + st);
        const int em = a.m_exp[b];
        const float um = em ? power_of_two(em) : 0.0f;
        const VUnit uv(a.v_exp[b]);
        decode_m(mc.x, um, m);
        decode_m(mc.y, um, m + 4);
        decode_v(vc.x, uv, v);
        decode_v(vc.y, uv, v + 4);
      } else {
        load_f32x8(static_cast<float*>(a.m) + st, m);
        load_f32x8(static_cast<float*>(a.v) + st, v);
      }
      const float keep = 1.0f - s.lr * t.decay;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] *= s.scale;
        m[k] = __fadd_rn(__fmul_rn(m[k], c.b1), __fmul_rn(g[k], c.c1));
        v[k] = __fadd_rn(__fmul_rn(v[k], c.b2), __fmul_rn(__fmul_rn(g[k], c.c2), g[k]));
        const float den = __fmaf_rn(sqrt_near(v[k]), s.root, a.eps);
        p[k] = __fmaf_rn(-s.size, m[k] * rcp_near(den), p[k] * keep);
      }
      if (!full)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= n) m[k] = v[k] = 0.0f;  // whatever a state that was handed in had there
      store8(t.p, at, p_type, whole, n, p);
      if (t.copy) store8(t.copy, at, copy_type, whole, n, p);
      if constexpr (EIGHT) {
        uint32_t tm = 0, tv = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          tm = max(tm, __float_as_uint(m[k]) & 0x7fffffffu);
          tv = max(tv, __float_as_uint(v[k]) & 0x7fffffffu);
        }
        tm = __reduce_max_sync(0xffffffffu, tm);
        tv = __reduce_max_sync(0xffffffffu, tv);
        // Nothing infinite, not a number or near the largest fp32 value: the usual case.
        const bool usual = max(tm, tv) < 0x7f000000u;
        if (!usual) {
          tm = tv = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t x = __float_as_uint(m[k]) & 0x7fffffffu, y = __float_as_uint(v[k]) & 0x7fffffffu;
            if (x < 0x7f800000u) tm = max(tm, x);
            if (y < 0x7f800000u) tv = max(tv, y);
          }
          tm = __reduce_max_sync(0xffffffffu, tm);
          tv = __reduce_max_sync(0xffffffffu, tv);
        }
        const int em = block_exp<7>(tm), ev = block_exp<23>(tv);
        const float upm = em ? power_of_two(254 - em) : 0.0f;
        const float upv = ev ? power_of_two(254 - ev) : 0.0f;
        uint32_t mo[2] = {0, 0}, vo[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint64_t call = st / 4 + h;
          const uint4 w = philox4x32_10(
              make_uint4((uint32_t)call, (uint32_t)(call >> 32), s.lo, s.hi), c.keys);
          uint32_t cm[4], cv[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t r = word_of(w, k), nm = (r << 4) & 0xffff0u, nv = (r >> 12) & 0xffff0u;
            const float x = m[4 * h + k];
            if (usual) {
              cm[k] = encode<7>(fabsf(x), upm, nm);
              cv[k] = encode<23>(v[4 * h + k], upv, nv);
            } else {
              cm[k] = encode_any<7>(fabsf(x), upm, nm);
              cv[k] = encode_any<23>(v[4 * h + k], upv, nv);
            }
            cm[k] |= (__float_as_uint(x) & 0x80000000u) >> 24;
          }
          mo[h] = __byte_perm(__byte_perm(cm[0], cm[1], 0x0040), __byte_perm(cm[2], cm[3], 0x0040), 0x5410);
          vo[h] = __byte_perm(__byte_perm(cv[0], cv[1], 0x0040), __byte_perm(cv[2], cv[3], 0x0040), 0x5410);
        }
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + st) = make_uint2(mo[0], mo[1]);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + st) = make_uint2(vo[0], vo[1]);
        if (lane == 0) {
          a.m_exp[b] = (uint8_t)em;
          a.v_exp[b] = (uint8_t)ev;
        }
      } else {
        store_f32x8(static_cast<float*>(a.m) + st, m);
        store_f32x8(static_cast<float*>(a.v) + st, v);
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
  using B = __nv_bfloat16;
  const uint2 mc = *reinterpret_cast<const uint2*>(m + st);
  const uint2 vc = *reinterpret_cast<const uint2*>(v + st);
  const int em = m_exp[b];
  const float um = em ? power_of_two(em) : 0.0f;
  const VUnit uv(v_exp[b]);
  float x[8];
  decode_m(mc.x, um, x);
  decode_m(mc.y, um, x + 4);
  *reinterpret_cast<uint4*>(m_out + st / 2) = pack8<B>(x);
  decode_v(vc.x, uv, x);
  decode_v(vc.y, uv, x + 4);
  *reinterpret_cast<uint4*>(v_out + st / 2) = pack8<B>(x);
}

template <int CAP>
cudaError_t launch(const AdamCall& c, const AdamTensor* t, cudaStream_t s) {
  AdamTable<CAP> table;
  auto lies = [](const void* p, int type) {
    return reinterpret_cast<uintptr_t>(p) % (type == OB_TYPE_F32 ? 32 : 16) == 0;
  };
  for (int i = 0; i < c.count; ++i) {
    table.t[i] = t[i];
    const bool whole = lies(t[i].p, t[i].types & 255) && lies(t[i].g, c.a.g_type) &&
                       lies(t[i].copy, t[i].types >> 8);
    table.t[i].types |= (int)whole << 16;
  }
  const uint64_t want = (c.blocks + kAdamThreads / 32 - 1) / (kAdamThreads / 32);
  const int grid = (int)(want < 1 ? 1 : want < kAdamGrid ? want : kAdamGrid);
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
