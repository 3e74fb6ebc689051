// Dropout with a mask that is never stored: y = residual + keep * x * scale.
//
// Two (with a residual three) streams of elements and one Philox call per
// eight of them: ten rounds of two wide products and two three-way xors, 72
// issue cycles of a scheduler for a warp's 256 elements.  Four schedulers of
// 152 SMs draw for 4.2e12 elements a second, where HBM brings at most 1.7e12
// of the smallest type: HBM is the bound (65536 x 2048 bf16 with a residual in
// 117.4 us, 6.86 TB/s; 16384 x 1024 in 18.5 us, 5.45 TB/s, the launch and the
// tail included).  Rows at any alignment into one aligned run are read in
// aligned words and shifted (65536 x 2001 bf16 with a residual in 180 us,
// 4.4 TB/s: the shifts and the rows' ends); other strides take an element a
// lane and step, where addresses and narrow accesses are the bound (429 us).
#include <type_traits>

#include "elem.cuh"
#include "keep.cuh"
#include "model.cuh"

namespace ob {
namespace {

constexpr int kDropThreads = 256;

// Eight elements in fp32, from and to 16-byte aligned memory.
template <typename T>
struct Eight {
  uint4 a[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) a[i] = __ldcs(q + i);
  }
  __device__ __forceinline__ void store(T* p) const {
    uint4* q = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) q[i] = a[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
      memcpy(v, a, 32);
    } else {
      const uint32_t w[4] = {a[0].x, a[0].y, a[0].z, a[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (sizeof(T) == 4)
      memcpy(a, v, 32);
    else
      a[0] = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                        pack2<T>(v[6], v[7]));
  }
};

__device__ __forceinline__ float drop1(float x, float r, bool keep, float scale) {
  return keep ? __fmaf_rn(x, scale, r) : r;
}

// Groups of eight that are 16-byte aligned in every array: one row, or rows
// of a multiple of eight elements whose starts are aligned.  A thread takes
// two groups a block apart, so that its loads and two Philox chains overlap.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) k_dropout_vec(const DropoutArgs a) {
  const uint64_t groups = (a.n + 7) / 8;
  const uint64_t g0 = (uint64_t)blockIdx.x * (2 * kDropThreads) + threadIdx.x;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  const uint64_t per_row = a.cols / 8;
  uint64_t xo[2], ro[2], yo[2];
  Eight<T> xv[2], rv[2];
  bool full[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint64_t g = g0 + (uint64_t)u * kDropThreads;
    if (a.rows == 1) {
      xo[u] = ro[u] = yo[u] = g * 8;
    } else {
      const uint64_t r = groups <= 0xffffffffull ? (uint32_t)g / (uint32_t)per_row : g / per_row;
      const uint64_t c = (g - r * per_row) * 8;
      xo[u] = r * a.ldx + c;
      ro[u] = r * a.ldr + c;
      yo[u] = r * a.ldy + c;
    }
    full[u] = g * 8 + 8 <= a.n;
    if (full[u]) {
      xv[u].load(x + xo[u]);
      if (RES) rv[u].load(res + ro[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint64_t g = g0 + (uint64_t)u * kDropThreads;
    if (g >= groups) break;
    uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (a.keep.T) w = keep_words(a.keep, g);
    if (full[u]) {
      float v[8], r[8];
      xv[u].get(v);
      if (RES) rv[u].get(r);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = drop1(v[i], RES ? r[i] : 0.0f, kept(w, i, a.keep.T), a.keep.scale);
      xv[u].set(v);
      xv[u].store(y + yo[u]);
    } else {  // the last group of one row
      const uint32_t b = keep_byte(w, a.keep.T);
      for (int i = 0; g * 8 + i < a.n; ++i)
        y[yo[u] + i] = from_f32<T>(drop1(to_f32(x[xo[u] + i]), RES ? to_f32(res[ro[u] + i]) : 0.0f,
                                         b >> i & 1, a.keep.scale));
    }
  }
}

// Eight elements from memory of any alignment: the 16-byte words that they lie
// in (each holds one of them at least), shifted into place.
template <typename T>
__device__ __forceinline__ void load_shifted(Eight<T>& to, const T* p) {
  constexpr int N = sizeof(T) / 2;
  const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
  const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - off);
  uint4 w[N + 1];
#pragma unroll
  for (int i = 0; i <= N; ++i) w[i] = i < N || off ? q[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) to.a[i] = shifted<T>(w[i], w[i + 1], off);
}

// Into one aligned run from rows at any alignment (a slice of a wider buffer):
// a thread takes an aligned eight of y (fp32 two, a block apart: 4099 x 1001
// 7.6 -> 6.7 us; with 2-byte types two cost 65536 x 2001 6%).  Eights that lie
// across a row's end are read one by one.
template <typename T>
constexpr int kRunEights = sizeof(T) / 2;
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) k_dropout_run(const DropoutArgs a) {
  constexpr int U = kRunEights<T>;
  const uint64_t g0 = (uint64_t)blockIdx.x * (U * kDropThreads) + threadIdx.x;
  float v[U][8], r[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t e0 = 8 * (g0 + u * kDropThreads);
    if (e0 >= a.n) break;
    const uint64_t row = a.small ? __umul64hi(e0, a.magic) : e0 / a.cols;
    uint64_t c = e0 - row * a.cols;
    const T* x = static_cast<const T*>(a.x) + row * a.ldx + c;
    const T* res = RES ? static_cast<const T*>(a.residual) + row * a.ldr + c : nullptr;
    if (c + 8 <= a.cols) {
      Eight<T> xv, rv;
      load_shifted(xv, x);
      if (RES) load_shifted(rv, res);
      xv.get(v[u]);
      if (RES) rv.get(r[u]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[u][k] = r[u][k] = 0.0f;
        if (e0 + k >= a.n) continue;
        v[u][k] = to_f32(*x++);
        if (RES) r[u][k] = to_f32(*res++);
        if (++c == a.cols) {
          c = 0;
          x += a.ldx - a.cols;
          if (RES) res += a.ldr - a.cols;
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t g = g0 + u * kDropThreads, e0 = 8 * g;
    if (e0 >= a.n) break;
    uint4 w = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (a.keep.T) w = keep_words(a.keep, g);
    float o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      o[k] = drop1(v[u][k], RES ? r[u][k] : 0.0f, kept(w, k, a.keep.T), a.keep.scale);
    T* y = static_cast<T*>(a.y) + e0;
    if (e0 + 8 <= a.n) {
      Eight<T> out;
      out.set(o);
      out.store(y);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (e0 + k < a.n) y[k] = from_f32<T>(o[k]);
    }
  }
}

// Any strides and alignment: a warp takes 256 elements, lane l draws the keep
// bits of its l-th eight, and in step k the lanes handle elements 32k..32k+31
// (consecutive addresses) with the bits fetched from the lane that drew them.
template <typename T, bool RES>
__global__ void __launch_bounds__(kDropThreads) k_dropout_any(const DropoutArgs a) {
  const int lane = threadIdx.x & 31;
  const uint64_t e0 =
      ((uint64_t)blockIdx.x * (kDropThreads / 32) + threadIdx.x / 32) * 256;
  if (e0 >= a.n) return;
  // The lane's first element; the next ones are 32 columns on, and where that
  // passes the end of a row, in the next.
  const uint64_t first = e0 + lane;
  uint64_t row = a.small ? __umul64hi(first, a.magic) : first / a.cols;
  if (a.cols == 1) row = first;
  uint64_t c = first - row * a.cols;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx + c;
  const T* res = RES ? static_cast<const T*>(a.residual) + row * a.ldr + c : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ldy + c;
  float v[8], r[8];
  T* to[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (first + 32 * k >= a.n) break;
    v[k] = to_f32(*x);
    r[k] = RES ? to_f32(*res) : 0.0f;
    to[k] = y;
    c += 32;
    uint32_t rows = 0;
    if (a.cols >= 32) {
      rows = c >= a.cols;
      if (rows) c -= a.cols;
    } else {
      rows = (uint32_t)c / (uint32_t)a.cols;
      c -= rows * (uint32_t)a.cols;
    }
    x += 32 + rows * (a.ldx - a.cols);
    if (RES) res += 32 + rows * (a.ldr - a.cols);
    y += 32 + rows * (a.ldy - a.cols);
  }
  uint32_t byte = 0xffu;
  if (a.keep.T) byte = keep_byte(keep_words(a.keep, e0 / 8 + lane), a.keep.T);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = __shfl_sync(0xffffffffu, byte, 4 * k + (lane >> 3));
    if (first + 32 * k < a.n)
      *to[k] = from_f32<T>(drop1(v[k], r[k], b >> (lane & 7) & 1, a.keep.scale));
  }
}

template <typename T>
cudaError_t launch(const DropoutArgs& a, cudaStream_t s) {
  auto aligned = [&](const void* p, uint64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.rows == 1 || ld % 8 == 0);
  };
  const bool vec = aligned(a.x, a.ldx) && aligned(a.y, a.ldy) &&
                   (!a.residual || aligned(a.residual, a.ldr)) &&
                   (a.rows == 1 || a.cols % 8 == 0);
  // Rows of less than eight make every eight cross one: 4000000 x 1 63 us, with
  // the kernel for any stride 45.  From eight on: 4099 x 1001 fp16 6.6 us
  // instead of 10.0, 65536 x 2001 bf16 with a residual 180 instead of 429.
  const bool run = !vec && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.cols >= 8 &&
                   (a.rows == 1 || a.ldy == a.cols);
  const uint64_t per = (vec ? 16ull : run ? 8ull * kRunEights<T> : 8ull) * kDropThreads;
  const dim3 grid((unsigned)((a.n + per - 1) / per));
  auto go = [&](auto with) {
    constexpr bool kRes = decltype(with)::value;
    if (vec)
      k_dropout_vec<T, kRes><<<grid, kDropThreads, 0, s>>>(a);
    else if (run)
      k_dropout_run<T, kRes><<<grid, kDropThreads, 0, s>>>(a);
    else
      k_dropout_any<T, kRes><<<grid, kDropThreads, 0, s>>>(a);
  };
  if (a.residual)
    go(std::true_type());
  else
    go(std::false_type());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int type, cudaStream_t s) {
  if (type == OB_TYPE_F32) return launch<float>(a, s);
  if (type == OB_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
  return launch<__half>(a, s);
}

}  // namespace ob
