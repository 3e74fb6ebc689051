// AdamW over many tensors, one launch for up to 128 of them.
//
// A warp takes blocks of 256 elements, eight of each a lane.  The table of
// tensors comes as the kernel's parameter: pointers may change from call to
// call, nothing is copied, and a graph keeps what it captured.
//
// Moments in 8 bits: a block's largest value gives its unit, a power of two, so
// that scaling is exact; a code is the value's bits in that unit, plus 16 random
// bits, cut off after three bits of significand.  The random bits are what lets
// v fall: 0.1% a step is far below half a code.
//
// Moments in 32 bits are bound by HBM (302M fp32 parameters, 28 bytes each, 1.25 ms, 6.8
// TB/s).  In 8 bits, 16 bytes with a bf16 gradient and copy, it is HBM and the issue of
// 540 instructions for a warp's 256 elements, 100 of them the generator's (268M 725 us,
// 5.9 TB/s); with bf16 parameters, 10 bytes, the latter (67M 181 us, 3.7 TB/s; one
// element off their boundary 239 us).
#include <cmath>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "philox.cuh"
#include "tc.cuh"

namespace ob {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamPer = 64;  // two whole sectors of units
constexpr int kAdamBlocks = 3, kAdamBlocks8 = 4;  // of an SM at a time

constexpr int kAdamMost = 128;  // tensors of a launch: 7 KB of parameters

struct AdamTable {
  AdamTensor t[kAdamMost];
};

struct AdamCall {
  AdamArgs a;
  PhiloxKeys keys;
  uint64_t first, blocks;  // of the state, in this launch
  int per;                 // of a block of threads at a time, 8 bits: kAdamPer or fewer
  int count, last;         // last: this launch advances the counter
  float b1, c1, b2, c2;    // c = 1 - b
  float one;               // 1: x * one + y is a sum that no product is drawn into
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
// Eight of v: as fp32 bits, twenty places up, a code is its value times 2^-104, below the
// normal range too.  `up` is 2^104 times the unit, as far as fp32 goes.
__device__ __forceinline__ void decode_v(const uint2& w, int e, float* v) {
  const float up = e ? power_of_two(min(e + 104, 254)) : 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t x = h ? w.y : w.x;
    v[4 * h] = __uint_as_float((x << 20) & 0x0ff00000u) * up;
    v[4 * h + 1] = __uint_as_float((x << 12) & 0x0ff00000u) * up;
    v[4 * h + 2] = __uint_as_float((x << 4) & 0x0ff00000u) * up;
    v[4 * h + 3] = __uint_as_float((x >> 4) & 0x0ff00000u) * up;
  }
  // rare: a code 255, and units above what fp32's powers reach with the 2^104
  const uint32_t not_number = ((~w.x - 0x01010101u) & w.x) | ((~w.y - 0x01010101u) & w.y);
  if ((not_number & 0x80808080u) || e > 150) {
    const float more = power_of_two(max(e + 104 - 254, 0) + 127);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] *= more;
      if (((k < 4 ? w.x : w.y) >> (8 * (k & 3)) & 255u) == 255u) v[k] = __uint_as_float(0x7fffffffu);
    }
  }
}

// E of a block whose largest finite value has bits `top`.
template <int BIAS>
__device__ __forceinline__ int block_exp(uint32_t top) {
  const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
  return top == 0 ? 0 : min(max(e, BIAS == 7 ? 1 : 3), 246);
}

// The code of x from bit 20 on (and its sign at bit 31): x in the block's unit times
// 2^(BIAS - 127) has a code's exponent as its own, and fp32's values below the normal
// range are those of the codes; cut off toward zero there.  The random bits are added
// four places up.  No value of a block passes the largest code, whose unit goes by them
// all.
__device__ __forceinline__ uint32_t encode(float x, float up, uint32_t noise) {
  return __float_as_uint(__fmul_rz(x, up)) + 16u * noise;
}
// 2^(BIAS - 127) over the unit of E, for E in [1, BIAS + 126]
template <int BIAS>
__device__ __forceinline__ float up_of(int e) {
  return power_of_two(127 + BIAS - e);
}
// The same for any x and E: what is not finite has the code after the last.
template <int BIAS>
__device__ __forceinline__ uint32_t encode_any(float size, int e, uint32_t noise) {
  constexpr uint32_t most = BIAS == 7 ? 126 : 254;
  if (!(size < INFINITY)) return most + 1;
  if (e == 0) return 0;
  const float y = size * power_of_two(254 - e);  // in its unit
  const uint32_t c = min(encode(y, power_of_two(BIAS), noise) >> 20, most);
  return BIAS == 7 || size == 0.0f ? c : max(c, 1u);
}
// Bytes of four.
__device__ __forceinline__ uint32_t bytes4(const uint32_t (&c)[4]) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
// Four of encode()'s as bytes, their upper halves two a word first.
__device__ __forceinline__ uint32_t codes_v(const uint32_t (&c)[4]) {
  const uint32_t a = __byte_perm(c[0], c[1], 0x7632) >> 4, b = __byte_perm(c[2], c[3], 0x7632) >> 4;
  return __byte_perm(a, b, 0x6420);
}
__device__ __forceinline__ uint32_t codes_m(const uint32_t (&c)[4]) {
  uint32_t a = __byte_perm(c[0], c[1], 0x7632), b = __byte_perm(c[2], c[3], 0x7632);
  a = (a >> 4 & 0x007f007fu) | (a >> 8 & 0x00800080u);
  b = (b >> 4 & 0x007f007fu) | (b >> 8 & 0x00800080u);
  return __byte_perm(a, b, 0x6420);
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

// Eight as they lie in memory (`raw[1]` for fp32 alone).
struct Raw {
  uint4 raw[2];
  // Of a warp's 256 elements at any alignment to the element: the aligned words that hold
  // them, the last of which a lane shares with the next one.
  __device__ __forceinline__ void load_shifted(const char* p, int type) {
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* q = reinterpret_cast<const uint4*>(p - off);
    raw[0] = q[0];
    if (type == OB_TYPE_F32) raw[1] = q[1];
    if (off == 0) return;
    if (type == OB_TYPE_F32) {
      raw[0] = shifted<float>(raw[0], raw[1], off);
      raw[1] = shifted<float>(raw[1], q[2], off);
    } else {
      raw[0] = shifted<__half>(raw[0], q[1], off);
    }
  }
  __device__ __forceinline__ void load(const void* p, int type) {
    if (type == OB_TYPE_F32) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(raw[0].x), "=r"(raw[0].y), "=r"(raw[0].z), "=r"(raw[0].w),
                     "=r"(raw[1].x), "=r"(raw[1].y), "=r"(raw[1].z), "=r"(raw[1].w)
                   : "l"(p));
    } else {
      raw[0] = *static_cast<const uint4*>(p);
    }
  }
  __device__ __forceinline__ void get(int type, float (&v)[8]) const {
    if (type == OB_TYPE_F32)
      memcpy(v, raw, 32);
    else if (type == OB_TYPE_BF16)
      unpack8<__nv_bfloat16>(raw[0], v);
    else
      unpack8<__half>(raw[0], v);
  }
};

// n of the eight from p on, which may lie anywhere.
__device__ __forceinline__ void load_any(const void* p, int type, int n, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = k < n ? load_as_f32(p, k, type) : 0.0f;
}
__device__ __forceinline__ void store_aligned(void* p, int type, const float (&v)[8]) {
  if (type == OB_TYPE_F32)
    store_f32x8(static_cast<float*>(p), v);
  else
    *static_cast<uint4*>(p) = type == OB_TYPE_BF16 ? pack8<__nv_bfloat16>(v) : pack8<__half>(v);
}
__device__ __forceinline__ uint4 next_lanes(const uint4& a) {
  return make_uint4(__shfl_down_sync(0xffffffffu, a.x, 1), __shfl_down_sync(0xffffffffu, a.y, 1),
                    __shfl_down_sync(0xffffffffu, a.z, 1), __shfl_down_sync(0xffffffffu, a.w, 1));
}
// A warp's 256 elements from element `at` of its lanes on: at any alignment in aligned words,
// made of a lane's end and the next one's beginning, and what is left at either end.
template <typename T>
__device__ __forceinline__ void store_any(T* p, const uint4 (&r)[sizeof(T) / 2]) {
  const int lane = threadIdx.x & 31;
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  constexpr int kWords = sizeof(T) / 2;
  const uint4 next = next_lanes(r[0]);
  char* q = reinterpret_cast<char*>(p) + (16 - off);
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    if (i + 1 < kWords || lane < 31)
      *reinterpret_cast<uint4*>(q + 16 * i) = shifted<T>(r[i], i + 1 < kWords ? r[i + 1] : next, 16 - off);
  const int head = (int)((16 - off) / sizeof(T)), last = 8 * (kWords - 1) / kWords;
  T v[8];
  memcpy(v, r, sizeof r);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (lane == 0 ? k < head : lane == 31 && k >= last + head) p[k] = v[k];
}
// full: all of the warp's elements are there; n: of this lane's.
__device__ __forceinline__ void store8(void* p, int type, bool full, int n, const float (&v)[8]) {
  const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
  if (!full) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store_from_f32(p, k, type, v[k]);
  } else if (type == OB_TYPE_F32) {
    uint4 r[2];
    memcpy(r, v, 32);
    if (off) {
      store_any(static_cast<float*>(p), r);
    } else {
      static_cast<uint4*>(p)[0] = r[0];
      static_cast<uint4*>(p)[1] = r[1];
    }
  } else {
    const uint4 r[1] = {type == OB_TYPE_BF16 ? pack8<__nv_bfloat16>(v) : pack8<__half>(v)};
    if (off)
      store_any(static_cast<__half*>(p), r);
    else
      *static_cast<uint4*>(p) = r[0];
  }
}

// The block that ends last has seen all others read the counter.
__device__ __forceinline__ void advance(const AdamCall& c, bool skip) {
  if (!c.last || skip) return;
  __syncthreads();
  if (threadIdx.x) return;
  unsigned* ticket = reinterpret_cast<unsigned*>(c.a.counter + 3);
  if (atomicAdd(ticket, 1u) == gridDim.x - 1) {
    *ticket = 0;
    c.a.counter[0] += 1.0;
    c.a.counter[1] *= c.a.b1;
    c.a.counter[2] *= c.a.b2;
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

// What a step needs of the whole call, by one thread a block.
__device__ __forceinline__ AdamStep make_step(const AdamArgs& a) {
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
  return s;
}

// m, v and p of eight elements, two an instruction.  Every operation of m and v is
// rounded on its own (the assembler makes a packed product and sum one multiply-add, but
// does not draw a product into a multiply-add).
__device__ __forceinline__ void update8(const AdamCall& c, const AdamStep& s, float keep,
                                        const float (&g)[8], float (&p)[8], float (&m)[8],
                                        float (&v)[8]) {
  const uint64_t scale2 = pair(s.scale, s.scale), b1 = pair(c.b1, c.b1), c1 = pair(c.c1, c.c1);
  const uint64_t b2 = pair(c.b2, c.b2), c2 = pair(c.c2, c.c2), root2 = pair(s.root, s.root);
  const uint64_t one = pair(c.one, c.one), eps2 = pair(c.a.eps, c.a.eps);
  const uint64_t keep2 = pair(keep, keep), size2 = pair(-s.size, -s.size);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t g2 = mul2(pair(g[k], g[k + 1]), scale2);
    const uint64_t m2 = fma2(mul2(pair(m[k], m[k + 1]), b1), one, mul2(g2, c1));
    const uint64_t v2 = fma2(mul2(pair(v[k], v[k + 1]), b2), one, mul2(mul2(g2, c2), g2));
    unpair(m2, &m[k], &m[k + 1]);
    unpair(v2, &v[k], &v[k + 1]);
    float d0, d1;
    unpair(fma2(pair(sqrt_near(v[k]), sqrt_near(v[k + 1])), root2, eps2), &d0, &d1);
    const uint64_t q2 = fma2(mul2(m2, pair(rcp_near(d0), rcp_near(d1))), size2,
                             mul2(pair(p[k], p[k + 1]), keep2));
    unpair(q2, &p[k], &p[k + 1]);
  }
}

// Codes of eight moments of a lane and the block's units; `st`: the lane's first element
// in the state.
__device__ __forceinline__ void encode8(const AdamCall& c, const AdamStep& s, uint64_t st,
                                        const float (&m)[8], const float (&v)[8], uint2* mc,
                                        uint2* vc, int* em, int* ev) {
  float xm = 0.0f, xv = 0.0f;  // the largest; a NaN comes through
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    xm = max_nan(xm, fabsf(m[k]));
    xv = max_nan(xv, v[k]);
  }
  const uint32_t tm = __reduce_max_sync(0xffffffffu, __float_as_uint(xm) & 0x7fffffffu);
  const uint32_t tv = __reduce_max_sync(0xffffffffu, __float_as_uint(xv) & 0x7fffffffu);
  *em = block_exp<7>(tm);
  *ev = block_exp<23>(tv);
  uint32_t mo[2], vo[2];
  const uint64_t call = st / 4;  // even
  uint4 r[2] = {make_uint4((uint32_t)call, (uint32_t)(call >> 32), s.lo, s.hi),
                make_uint4((uint32_t)call + 1, (uint32_t)(call >> 32), s.lo, s.hi)};
  philox4x32_10_x2(r[0], r[1], c.keys);
  // Units that one product reaches (m below 2^13, v below 2^29), nothing but numbers.
  if (tm < 0x46000000u && tv < 0x4e000000u && tm && tv) {
    const float upm = up_of<7>(*em), upv = up_of<23>(*ev);
    uint32_t cm[2][4], cv[2][4], none = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = word_of(r[h], k);
        cm[h][k] = encode(m[4 * h + k], upm, x & 0xffffu);
        cv[h][k] = encode(v[4 * h + k], upv, x >> 16);
      }
      mo[h] = codes_m(cm[h]);
      vo[h] = codes_v(cv[h]);
      none |= (vo[h] - 0x01010101u) & ~vo[h];
    }
    if (none & 0x80808080u)  // a byte of 0 is rare, and of a positive v it becomes 1
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (cv[k / 4][k % 4] >> 20 == 0 && v[k] > 0.0f) vo[k / 4] |= 1u << (8 * (k % 4));
  } else {
    uint32_t fm = 0, fv = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t x = __float_as_uint(m[k]) & 0x7fffffffu, y = __float_as_uint(v[k]) & 0x7fffffffu;
      if (x < 0x7f800000u) fm = max(fm, x);
      if (y < 0x7f800000u) fv = max(fv, y);
    }
    *em = block_exp<7>(__reduce_max_sync(0xffffffffu, fm));
    *ev = block_exp<23>(__reduce_max_sync(0xffffffffu, fv));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t cm[4], cv[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = word_of(r[h], k);
        const float mk = m[4 * h + k];
        cm[k] = encode_any<7>(fabsf(mk), *em, x & 0xffffu) |
                (__float_as_uint(mk) & 0x80000000u) >> 24;
        cv[k] = encode_any<23>(v[4 * h + k], *ev, x >> 16);
      }
      mo[h] = bytes4(cm);
      vo[h] = bytes4(cv);
    }
  }
  *mc = make_uint2(mo[0], mo[1]);
  *vc = make_uint2(vo[0], vo[1]);
}

// A block of the state on its way, and a lane's part of it.
struct Work {
  bool any;          // there is a gradient
  bool full;         // all of it is the tensor's
  bool aligned;      // full, and p, copy and gradient lie on 32 bytes, or 16 of 2-byte types
  int n;             // elements of this lane
  int types;
  uint64_t st;       // the lane's first element in the state
  char *p, *g, *copy;  // at that element; copy: or null
  float keep;
};

// Finds the tensors of a warp's blocks, which come in order.
struct Walk {
  int tensor;
  __device__ __forceinline__ Work take(const AdamCall& c, const AdamTable& table, float lr,
                                       uint64_t b) {
    const int lane = threadIdx.x & 31;
    while (tensor + 1 < c.count && table.t[tensor + 1].first <= b) ++tensor;
    const AdamTensor& t = table.t[tensor];
    Work w;
    w.any = t.g != nullptr;
    const uint64_t begin = (b - t.first) * kAdamBlock, at = begin + lane * 8;
    w.full = begin + kAdamBlock <= t.n;
    w.aligned = w.full && t.types >> 16;
    w.n = w.full ? 8 : at < t.n ? (int)min((uint64_t)8, t.n - at) : 0;
    w.types = t.types;
    w.st = b * kAdamBlock + lane * 8;
    w.p = static_cast<char*>(t.p) + (at << ((t.types & 255) == OB_TYPE_F32 ? 2 : 1));
    w.g = static_cast<char*>(const_cast<void*>(t.g)) + (at << (c.a.g_type == OB_TYPE_F32 ? 2 : 1));
    w.copy = nullptr;
    if (t.copy)
      w.copy = static_cast<char*>(t.copy) + (at << ((t.types >> 8 & 255) == OB_TYPE_F32 ? 2 : 1));
    w.keep = 1.0f - lr * t.decay;
    return w;
  }
};

// Moments in 8 bits.  P, G: the types of p (-1: by the tensor) and of the gradients.  A
// block of threads takes `per` blocks of the state at a time, whose units it reads and
// writes together: a byte at a time, from warps all over the card, they cost a quarter of
// the whole time (268M elements 704 -> 884 us).
template <int P, int G>
__global__ void __launch_bounds__(kAdamThreads, kAdamBlocks8)
    k_adamw8(const __grid_constant__ AdamCall c, const __grid_constant__ AdamTable table) {
  __shared__ uint8_t units[2 * kAdamPer];  // of m, then of v
  __shared__ AdamStep shared_step;
  const AdamArgs& a = c.a;
  if (threadIdx.x == 0) shared_step = make_step(a);
  __syncthreads();
  const AdamStep s = shared_step;
  const int lane = threadIdx.x & 31;
  uint8_t *ms = static_cast<uint8_t*>(a.m), *vs = static_cast<uint8_t*>(a.v);
  const int warp = threadIdx.x >> 5, tid = threadIdx.x;
  const uint64_t end = c.first + c.blocks, chunk0 = c.first / c.per;
  Walk walk{0};
  uint64_t b0 = 0, b1 = 0;  // of the chunk before, then of this one
  for (uint64_t k = blockIdx.x; !s.skip; k += gridDim.x) {
    uint8_t* mine = (tid < kAdamPer ? a.m_exp : a.v_exp) + (tid & (kAdamPer - 1));
    if (tid < 2 * kAdamPer && b0 + (tid & (kAdamPer - 1)) < b1) mine[b0] = units[tid];
    b0 = max(c.first, (chunk0 + k) * c.per);
    b1 = min(end, (chunk0 + k + 1) * c.per);
    if (b0 >= end) break;
    if (tid < 2 * kAdamPer && b0 + (tid & (kAdamPer - 1)) < b1) units[tid] = mine[b0];
    __syncthreads();
    for (uint64_t b = b0 + warp; b < b1; b += kAdamThreads / 32) {
      const Work w = walk.take(c, table, s.lr, b);
      if (!w.any) continue;
      const int p_type = P < 0 ? w.types & 255 : P;
      const uint2 wm = *reinterpret_cast<const uint2*>(ms + w.st);
      const uint2 wv = *reinterpret_cast<const uint2*>(vs + w.st);
      const int wem = units[b - b0], wev = units[kAdamPer + b - b0];
      float g[8], p[8], m[8], v[8];
      if (w.full) {
        Raw gr, pr;
        if (w.aligned) {
          gr.load(w.g, G);
          pr.load(w.p, p_type);
        } else {
          gr.load_shifted(w.g, G);
          pr.load_shifted(w.p, p_type);
        }
        gr.get(G, g);
        pr.get(p_type, p);
      } else {
        load_any(w.g, G, w.n, g);
        load_any(w.p, p_type, w.n, p);
      }
      const float um = wem ? power_of_two(wem) : 0.0f;
      decode_m(wm.x, um, m);
      decode_m(wm.y, um, m + 4);
      decode_v(wv, wev, v);
      update8(c, s, w.keep, g, p, m, v);
      if (!w.full)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= w.n) m[k] = v[k] = 0.0f;  // whatever a state that was handed in had there
      if (w.aligned) {
        store_aligned(w.p, p_type, p);
        if (w.copy) store_aligned(w.copy, w.types >> 8 & 255, p);
      } else {
        store8(w.p, p_type, w.full, w.n, p);
        if (w.copy) store8(w.copy, w.types >> 8 & 255, w.full, w.n, p);
      }
      uint2 mo, vo;
      int em, ev;
      encode8(c, s, w.st, m, v, &mo, &vo, &em, &ev);
      *reinterpret_cast<uint2*>(ms + w.st) = mo;
      *reinterpret_cast<uint2*>(vs + w.st) = vo;
      if (lane == 0) {
        units[b - b0] = (uint8_t)em;
        units[kAdamPer + b - b0] = (uint8_t)ev;
      }
    }
    __syncthreads();
  }
  advance(c, s.skip);
}

// Moments in 32 bits: HBM bounds it, whatever the types.
__global__ void __launch_bounds__(kAdamThreads, kAdamBlocks)
    k_adamw32(const __grid_constant__ AdamCall c, const __grid_constant__ AdamTable table) {
  __shared__ AdamStep shared_step;
  const AdamArgs& a = c.a;
  if (threadIdx.x == 0) shared_step = make_step(a);
  __syncthreads();
  const AdamStep s = shared_step;
  const int lane = threadIdx.x & 31;
  if (!s.skip) {
    Walk walk{0};
    for (uint64_t i = (uint64_t)blockIdx.x * (kAdamThreads / 32) + (threadIdx.x >> 5); i < c.blocks;
         i += (uint64_t)gridDim.x * (kAdamThreads / 32)) {
      const Work w = walk.take(c, table, s.lr, c.first + i);
      if (!w.any) continue;
      float g[8], p[8], m[8], v[8];
      const int p_type = w.types & 255;
      load_f32x8(static_cast<float*>(a.m) + w.st, m);
      load_f32x8(static_cast<float*>(a.v) + w.st, v);
      if (w.full) {
        Raw pr, gr;
        if (w.aligned) {
          gr.load(w.g, a.g_type);
          pr.load(w.p, p_type);
        } else {
          gr.load_shifted(w.g, a.g_type);
          pr.load_shifted(w.p, p_type);
        }
        gr.get(a.g_type, g);
        pr.get(p_type, p);
      } else {
        load_any(w.g, a.g_type, w.n, g);
        load_any(w.p, p_type, w.n, p);
      }
      update8(c, s, w.keep, g, p, m, v);
      if (!w.full)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k >= w.n) m[k] = v[k] = 0.0f;
      if (w.aligned) {
        store_aligned(w.p, p_type, p);
        if (w.copy) store_aligned(w.copy, w.types >> 8 & 255, p);
      } else {
        store8(w.p, p_type, w.full, w.n, p);
        if (w.copy) store8(w.copy, w.types >> 8 & 255, w.full, w.n, p);
      }
      store_f32x8(static_cast<float*>(a.m) + w.st, m);
      store_f32x8(static_cast<float*>(a.v) + w.st, v);
    }
  }
  advance(c, s.skip);
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
  float x[8];
  decode_m(mc.x, um, x);
  decode_m(mc.y, um, x + 4);
  *reinterpret_cast<uint4*>(m_out + st / 2) = pack8<B>(x);
  decode_v(vc, v_exp[b], x);
  *reinterpret_cast<uint4*>(v_out + st / 2) = pack8<B>(x);
}

template <int P>
void launch8(const AdamCall& c, const AdamTable& table, int grid, cudaStream_t s) {
  if (c.a.g_type == OB_TYPE_F32)
    k_adamw8<P, OB_TYPE_F32><<<grid, kAdamThreads, 0, s>>>(c, table);
  else if (c.a.g_type == OB_TYPE_BF16)
    k_adamw8<P, OB_TYPE_BF16><<<grid, kAdamThreads, 0, s>>>(c, table);
  else
    k_adamw8<P, OB_TYPE_F16><<<grid, kAdamThreads, 0, s>>>(c, table);
}

cudaError_t launch(const AdamCall& call, const AdamTensor* t, cudaStream_t s) {
  AdamCall c = call;
  AdamTable table;
  auto lies = [](const void* p, int type) {
    return reinterpret_cast<uintptr_t>(p) % (type == OB_TYPE_F32 ? 32 : 16) == 0;
  };
  int p_type = c.count ? t[0].types & 255 : 0;
  for (int i = 0; i < c.count; ++i) {
    table.t[i] = t[i];
    const bool aligned = lies(t[i].p, t[i].types & 255) && lies(t[i].g, c.a.g_type) &&
                         lies(t[i].copy, t[i].types >> 8);
    table.t[i].types |= (int)aligned << 16;
    if ((t[i].types & 255) != p_type) p_type = -1;
  }
  const uint64_t most = (c.a.bits == 8 ? kAdamBlocks8 : kAdamBlocks) * 152;  // all that run at a time
  // Few blocks are spread over the card, a warp one of them.
  c.per = c.a.bits == 8 && c.blocks >= most * kAdamPer ? kAdamPer : kAdamThreads / 32;
  const uint64_t want = c.blocks ? (c.first + c.blocks - 1) / c.per - c.first / c.per + 1 : 1;
  const int grid = (int)(want < most ? want : most);
  if (c.a.bits == 32)
    k_adamw32<<<grid, kAdamThreads, 0, s>>>(c, table);
  else if (p_type == OB_TYPE_F32)
    launch8<OB_TYPE_F32>(c, table, grid, s);
  else if (p_type == OB_TYPE_BF16)
    launch8<OB_TYPE_BF16>(c, table, grid, s);
  else if (p_type == OB_TYPE_F16)
    launch8<OB_TYPE_F16>(c, table, grid, s);
  else
    launch8<-1>(c, table, grid, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_adamw(const AdamArgs& a, const AdamTensor* t, int count, cudaStream_t s) {
  AdamCall c{};
  c.a = a;
  c.keys = philox_keys((uint32_t)a.seed, (uint32_t)(a.seed >> 32));
  c.b1 = (float)a.b1;
  c.c1 = (float)(1.0 - a.b1);
  c.b2 = (float)a.b2;
  c.c2 = (float)(1.0 - a.b2);
  c.one = 1.0f;
  int at = 0;
  do {
    c.count = count - at < kAdamMost ? count - at : kAdamMost;
    c.last = at + c.count == count;
    c.first = c.count ? t[at].first : 0;
    c.blocks = 0;
    if (c.count) {
      const AdamTensor& end = t[at + c.count - 1];
      c.blocks = end.first + (end.n + kAdamBlock - 1) / kAdamBlock - c.first;
    }
    const cudaError_t e = launch(c, t + at, s);
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
