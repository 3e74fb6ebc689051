// The dense layer: y = act(x w^T + b) + residual and its gradients.  The
// products are k_gemm.cu's; here is what is around them.
//
// dz = dy act'(z) is made once, as the operand of both products of the backward
// pass, and summed down the columns on the way: each block adds its share of
// the rows, a second kernel the blocks' sums in their order.  HBM bounds it, and the
// slope's arithmetic near to it (16384 x 4096 bf16 with GELU 74 us for 403 MB, 5.4 TB/s; making it
// inside the products would do its arithmetic once for every 256 columns of dx).
//
// Copies by TMA want 16-byte boundaries: matrices that lie elsewhere are first
// copied into the workspace, their rows padded to multiples of 16 bytes (the
// products' time is many times that of the copy).
#include <type_traits>

#include "act.cuh"
#include "elem.cuh"
#include "layers.cuh"
#include "model.cuh"

namespace ob {
namespace {

constexpr int kDzThreads = 128;
constexpr int kDzBlocks = 5;  // of an SM at a time

struct DzArgs {
  Mat dy, z, dz;      // dz: data or null
  float* partial;     // [parts][N], or null
  int64_t M, N;
  int parts, tx;      // threads of a block along the columns, a power of two
  int act;
};

// V elements as they lie in memory (8: 16 bytes).
template <typename T, int V>
struct Cell {
  T v[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      memcpy(v, &u, 16);
    } else {
      v[0] = *p;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (V == 8) {
      uint4 u;
      memcpy(&u, v, 16);
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      *p = v[0];
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f32(v[k]);
  }
  __device__ __forceinline__ void put(const float (&f)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = from_f32<T>(f[k]);
  }
};

// V columns a thread (8: 16-byte loads).
template <typename T, int V>
__global__ void __launch_bounds__(kDzThreads, kDzBlocks) k_dz(const __grid_constant__ DzArgs a) {
  __shared__ float sums[kDzThreads * V];
  grid_wait();
  const int x = threadIdx.x & (a.tx - 1), y = threadIdx.x / a.tx, ty = kDzThreads / a.tx;
  const int64_t n = ((int64_t)blockIdx.x * a.tx + x) * V;
  const int64_t per = (a.M + a.parts - 1) / a.parts;
  const int64_t r0 = (int64_t)blockIdx.y * per, r1 = r0 + per < a.M ? r0 + per : a.M;
  float acc[V];
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.0f;
  if (n < a.N)
    by_act(a.act, [&](auto act) {
      constexpr int kAct = decltype(act)::value;
      // Several rows' loads are on their way at once: the stores, which may touch anything as
      // far as the compiler knows, come behind them.
      constexpr int B = 4;
      for (int64_t r = r0 + y; r < r1; r += B * ty) {
        Cell<T, V> dy[B], z[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (r + b * ty < r1) {
            dy[b].load(static_cast<const T*>(a.dy.data) + (r + b * ty) * a.dy.ld + n);
            if (kAct != OB_ACT_NONE)
              z[b].load(static_cast<const T*>(a.z.data) + (r + b * ty) * a.z.ld + n);
          }
#pragma unroll
        for (int b = 0; b < B; ++b) {
          if (r + b * ty >= r1) break;
          float g[V], s[V];
          dy[b].get(g);
          if (kAct != OB_ACT_NONE) {
            z[b].get(s);
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] *= act_slope<kAct>(s[k]);
          }
#pragma unroll
          for (int k = 0; k < V; ++k) acc[k] += g[k];
          if (a.dz.data) {
            dy[b].put(g);
            dy[b].store(static_cast<T*>(a.dz.data) + (r + b * ty) * a.dz.ld + n);
          }
        }
      }
    });
  if (!a.partial) return;
#pragma unroll
  for (int k = 0; k < V; ++k) sums[threadIdx.x * V + k] = acc[k];
  __syncthreads();
  // a column a thread; its rows' sums in their order
  for (int c = threadIdx.x; c < a.tx * V; c += kDzThreads) {
    const int64_t col = (int64_t)blockIdx.x * a.tx * V + c;
    if (col >= a.N) break;
    float t = 0.0f;
    for (int q = 0; q < ty; ++q) t += sums[q * a.tx * V + c];
    a.partial[(int64_t)blockIdx.y * a.N + col] = t;
  }
}

// dbias from the parts: 32 columns a block, a warp every 32nd part.
template <typename T>
__global__ void __launch_bounds__(1024) k_dbias(const float* partial, int parts, int64_t N, T* out) {
  __shared__ float sums[32][32];
  grid_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (n < N)
#pragma unroll 8
    for (int p = w; p < parts; p += 32) t += partial[(int64_t)p * N + n];
  sums[w][lane] = t;
  __syncthreads();
  if (w || n >= N) return;
  t = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) t += sums[k][lane];
  out[n] = from_f32<T>(t);
}

// Copies of matrices that lie anywhere, rows padded to whole 16-byte words: a word a thread,
// from the two words that hold its bytes.
struct Realign {
  const char* from;
  char* to;
  int64_t rows, cols, ld, words;  // words of a padded row
  int64_t first;                  // its first thread
};
struct Realigns {
  Realign m[2];
  int count;
  int64_t threads;
};
__global__ void __launch_bounds__(256) k_realign(const __grid_constant__ Realigns a) {
  grid_wait();
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < a.threads; t += (int64_t)gridDim.x * 256) {
    const Realign& m = a.m[a.count > 1 && t >= a.m[1].first ? 1 : 0];
    const int64_t i = t - m.first, row = i / m.words, w = i - row * m.words;
    const char* begin = m.from + row * m.ld * 2;
    const char* p = begin + 16 * w;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* q = reinterpret_cast<const uint4*>(p - off);
    uint4 x = q[0];
    if (off) {
      const bool more = reinterpret_cast<const char*>(q + 1) < begin + 2 * m.cols;
      x = shifted<__half>(x, more ? q[1] : make_uint4(0, 0, 0, 0), off);
    }
    *reinterpret_cast<uint4*>(m.to + (row * m.words + w) * 16) = x;
  }
}

int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool by_tma(const Mat& m) { return on(m.data, 16) && m.ld % 8 == 0; }

int tiled(const Epilogue& e) {
  bool all = !e.bias || on(e.bias, 16);
  for (const Mat* m : {&e.out, &e.z, &e.residual}) all = all && (!m->data || by_tma(*m));
  return all;
}

int power_of_two(int64_t n, int most) {
  int p = 1;
  while (p < n && p < most) p *= 2;
  return p;
}

// Blocks along the rows of dz, by sizes alone (the workspace goes by it): eight
// rows a thread at least, and all that run at a time.
int dz_parts(int64_t M, int64_t N) {
  if (N == 0) return 1;
  const int tx = power_of_two((N + 7) / 8, kDzThreads);
  const int64_t columns = (N + 8 * tx - 1) / (8 * tx), rows = 8 * (kDzThreads / tx);
  int64_t most = kDzBlocks * 152 / columns;
  if (most < 1) most = 1;
  const int64_t parts = (M + rows - 1) / rows;
  return (int)(parts < 1 ? 1 : parts < most ? parts : most);
}

struct Area {  // the workspace, handed out in order
  uint8_t* base;
  size_t used;
  void* take(size_t bytes) {
    void* p = base + used;
    used += up256(bytes);
    return p;
  }
};

size_t mat_bytes(int64_t rows, int64_t cols) { return up256((size_t)(rows * padded(cols)) * 2); }

// Has m copied where its rows do not lie on 16 bytes.
void realign(Realigns* all, Mat* m, int64_t rows, int64_t cols, Area* area) {
  if (rows == 0 || cols == 0 || by_tma(*m)) return;
  void* to = area->take(mat_bytes(rows, cols));
  all->m[all->count++] = Realign{static_cast<const char*>(m->data), static_cast<char*>(to), rows, cols,
                                 m->ld, padded(cols) / 8, all->threads};
  all->threads += rows * (padded(cols) / 8);
  *m = Mat{to, padded(cols)};
}
cudaError_t launch(const Realigns& all, cudaStream_t s) {
  if (!all.count) return cudaSuccess;
  const int64_t blocks = (all.threads + 255) / 256;
  return launch_behind(k_realign, dim3((unsigned)(blocks < 152 * 16 ? blocks : 152 * 16)), dim3(256), 0,
                       s, all);
}

template <typename T>
cudaError_t make_dz(const DzArgs& d, bool wide, cudaStream_t s) {
  DzArgs a = d;
  const int V = wide ? 8 : 1;
  a.tx = power_of_two((a.N + V - 1) / V, kDzThreads);
  const dim3 grid((unsigned)((a.N + (int64_t)a.tx * V - 1) / ((int64_t)a.tx * V)), a.parts);
  return wide ? launch_behind(k_dz<T, 8>, grid, dim3(kDzThreads), 0, s, a)
              : launch_behind(k_dz<T, 1>, grid, dim3(kDzThreads), 0, s, a);
}

}  // namespace

size_t linear_workspace_bytes(const LinearArgs& a, bool backward) {
  const int64_t M = a.M, N = a.N, K = a.K, wr = a.w_kn ? K : N, wc = a.w_kn ? N : K;
  size_t b = a.unaligned ? mat_bytes(M, K) + mat_bytes(wr, wc) : 0;
  if (!backward) return b + up256(gemm_partial_bytes(M, N, K, false, false));
  if (a.act != OB_ACT_NONE || a.unaligned) b += mat_bytes(M, N);
  b += up256((size_t)dz_parts(M, N) * N * sizeof(float));
  const size_t p = gemm_partial_bytes(M, K, N, false, true);
  const size_t q = gemm_partial_bytes(wr, wc, M, true, true);
  return b + up256(p) + up256(q);
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s) {
  Area area{a.workspace, 0};
  Gemm g{};
  g.a = a.x;
  g.b = a.w;
  Realigns all{};
  realign(&all, &g.a, a.M, a.K, &area);
  realign(&all, &g.b, a.w_kn ? a.K : a.N, a.w_kn ? a.N : a.K, &area);
  const cudaError_t e = launch(all, s);
  if (e != cudaSuccess) return e;
  g.b_mn = a.w_kn;
  g.M = a.M;
  g.N = a.N;
  g.K = a.K;
  g.ep.bias = a.bias;
  g.ep.residual = a.residual;
  g.ep.z = a.z;
  g.ep.out = a.y;
  g.ep.act = a.act;
  g.ep.type = a.type;
  g.ep.tiled = tiled(g.ep);
  g.partial = static_cast<float*>(area.take(0));
  return launch_gemm(g, s);
}

cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t s) {
  Area area{a.workspace, 0};
  const int64_t M = a.M, N = a.N, K = a.K, wr = a.w_kn ? K : N, wc = a.w_kn ? N : K;
  const bool products = a.dx.data || a.dw.data;
  cudaError_t e = cudaSuccess;
  Mat dz = a.dy;
  DzArgs d{};
  const bool make = products && M > 0 && N > 0 && (a.act != OB_ACT_NONE || !by_tma(a.dy));
  if (make) {
    dz = Mat{area.take(mat_bytes(M, N)), padded(N)};
    d.dz = dz;
  }
  if (a.dbias) d.partial = static_cast<float*>(area.take((size_t)dz_parts(M, N) * N * sizeof(float)));
  if (make || a.dbias) {
    d.dy = a.dy;
    d.z = a.z;
    d.M = M;
    d.N = N;
    d.act = a.act;
    d.parts = dz_parts(M, N);
    const bool wide = N % 8 == 0 && by_tma(a.dy) && (a.act == OB_ACT_NONE || by_tma(a.z));
    e = a.type == OB_TYPE_BF16 ? make_dz<__nv_bfloat16>(d, wide, s) : make_dz<__half>(d, wide, s);
    if (e == cudaSuccess && a.dbias) {
      const dim3 grid((unsigned)((N + 31) / 32));
      e = a.type == OB_TYPE_BF16
              ? launch_behind(k_dbias<__nv_bfloat16>, grid, dim3(1024), 0, s, d.partial, d.parts, N,
                              static_cast<__nv_bfloat16*>(a.dbias))
              : launch_behind(k_dbias<__half>, grid, dim3(1024), 0, s, d.partial, d.parts, N,
                              static_cast<__half*>(a.dbias));
    }
  }
  Mat x = a.x, w = a.w;
  Realigns all{};
  if (a.dw.data) realign(&all, &x, M, K, &area);
  if (a.dx.data) realign(&all, &w, wr, wc, &area);
  if (e == cudaSuccess) e = launch(all, s);
  if (e != cudaSuccess) return e;
  Gemm g{}, h{};
  if (a.dw.data) {  // dw[n][k] = sum over m of dz(m, n) x(m, k), or turned
    g.a = a.w_kn ? x : dz;
    g.b = a.w_kn ? dz : x;
    g.a_mn = g.b_mn = 1;
    g.M = wr;
    g.N = wc;
    g.K = M;
    g.ep.out = a.dw;
  }
  if (a.dx.data) {  // dx[m][k] = sum over n of dz(m, n) w(n, k)
    h.a = dz;
    h.b = w;
    h.b_mn = !a.w_kn;
    h.M = M;
    h.N = K;
    h.K = N;
    h.ep.out = a.dx;
  }
  for (Gemm* p : {&g, &h}) {
    p->ep.type = a.type;
    p->ep.act = OB_ACT_NONE;
    p->pair = 1;
    p->ep.tiled = tiled(p->ep);
    p->partial = static_cast<float*>(area.take(gemm_partial_bytes(p->M, p->N, p->K, p->a_mn, p->pair)));
  }
  return launch_gemms(g, h, s);
}

}  // namespace ob
