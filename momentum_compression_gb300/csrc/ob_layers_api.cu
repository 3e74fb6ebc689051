// C entry points of layer norm, the dense layer and AdamW over many tensors
// (declared in ob.h).  Arguments are checked on the host before any CUDA call.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "layers.cuh"
#include "ob_internal.cuh"

namespace {

ob_status failf(ob_status st, const char* fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return ob::ctx_fail(nullptr, st, buf);
}

ob_status launched(cudaError_t e, const char* what) {
  if (e != cudaSuccess) return failf(OB_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return OB_OK;
}

bool known_type(int t) { return t == OB_TYPE_F32 || t == OB_TYPE_BF16 || t == OB_TYPE_F16; }
size_t type_bytes(int t) { return t == OB_TYPE_F32 ? 4 : 2; }

ob_status check_ptr(const void* p, size_t align, const char* name) {
  if (!p) return failf(OB_ERR_INVALID, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return failf(OB_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
  return OB_OK;
}
#define OB_TRY(call)                    \
  do {                                  \
    if (ob_status st_ = (call)) return st_; \
  } while (0)

ob_status check_sizes(size_t rows, size_t cols) {
  if (cols >= (1u << 24)) return failf(OB_ERR_INVALID, "cols = %zu must be below 2^24", cols);
  if (cols && rows > (1ull << 40) / cols)
    return failf(OB_ERR_INVALID, "%zu rows of %zu are over 2^40 elements", rows, cols);
  return OB_OK;
}

ob_status check_rows(const void* p, size_t ld, size_t rows, size_t cols, int type,
                     const char* name) {
  OB_TRY(check_ptr(p, type_bytes(type), name));
  if (rows > 1 && (ld < cols || ld >= (1ull << 40)))
    return failf(OB_ERR_INVALID, "%s: rows of %zu elements start %zu apart", name, cols, ld);
  return OB_OK;
}

size_t layernorm_partials(size_t rows, size_t cols) {
  return (size_t)ob::layernorm_bwd_parts(rows, (int)cols) * 2 * cols * sizeof(float);
}

constexpr int64_t kMost = 1ll << 30;

ob_status check_linear(const ob_linear* l) {
  if (!l) return failf(OB_ERR_INVALID, "linear is NULL");
  if (l->type != OB_TYPE_BF16 && l->type != OB_TYPE_F16)
    return failf(OB_ERR_UNSUPPORTED, "type = %d: linear takes OB_TYPE_BF16 and OB_TYPE_F16",
                 l->type);
  if (l->act < OB_ACT_NONE || l->act > OB_ACT_GELU_TANH)
    return failf(OB_ERR_INVALID, "act = %d is not an OB_ACT", l->act);
  if (l->M < 0 || l->N < 0 || l->K < 0 || l->M >= kMost || l->N >= kMost || l->K >= kMost)
    return failf(OB_ERR_INVALID, "M = %lld, N = %lld, K = %lld must be in [0, 2^30)",
                 (long long)l->M, (long long)l->N, (long long)l->K);
  const int64_t most = 1ll << 40;
  if (l->M * l->N > most || l->M * l->K > most || l->N * l->K > most)
    return failf(OB_ERR_INVALID, "M = %lld, N = %lld, K = %lld: a matrix is over 2^40 elements",
                 (long long)l->M, (long long)l->N, (long long)l->K);
  return OB_OK;
}

// A matrix of [rows][cols]; nothing is read or written where it is empty.
ob_status check_matrix(const ob_linear& l, const ob_matrix* m, int64_t rows, int64_t cols,
                       const char* name, ob::Mat* out) {
  *out = ob::Mat{nullptr, cols};
  if (!m) return failf(OB_ERR_INVALID, "%s is NULL", name);
  if (rows == 0 || cols == 0) {
    out->data = m->data;
    return OB_OK;
  }
  OB_TRY(check_ptr(m->data, 2, name));
  out->data = m->data;
  if (rows > 1) {
    if (m->ld < cols || m->ld >= (1ll << 37))
      return failf(OB_ERR_INVALID, "%s: ld = %lld must be in [%lld, 2^37)", name,
                   (long long)m->ld, (long long)cols);
    out->ld = m->ld;
  } else {
    out->ld = (cols + 7) / 8 * 8;
  }
  if (!l.unaligned) {
    OB_TRY(check_ptr(m->data, 16, name));
    if (out->ld % 8)
      return failf(OB_ERR_ALIGN, "%s: ld = %lld is not a multiple of 8", name,
                   (long long)out->ld);
  }
  return OB_OK;
}

ob::LinearArgs linear_args(const ob_linear& l) {
  ob::LinearArgs a{};
  a.type = l.type;
  a.act = l.act;
  a.w_kn = l.w_kn != 0;
  a.unaligned = l.unaligned != 0;
  a.M = l.M;
  a.N = l.N;
  a.K = l.K;
  return a;
}

ob_status check_workspace(const void* workspace, size_t have, size_t need, size_t align) {
  if (!need) return OB_OK;
  OB_TRY(check_ptr(workspace, align, "workspace"));
  if (have < need)
    return failf(OB_ERR_INVALID, "workspace of %zu bytes, %zu are needed", have, need);
  return OB_OK;
}

}  // namespace

extern "C" {

ob_status ob_layernorm_fwd(const void* x, size_t ldx, const void* residual, size_t ldr,
                           const void* weight, const void* bias, int w_type, void* y, size_t ldy,
                           void* sum, size_t lds, float* mean, float* rstd, size_t rows,
                           size_t cols, int type, double eps, ob_stream_t stream) {
  OB_TRACE();
  if (!known_type(type) || !known_type(w_type))
    return failf(OB_ERR_INVALID, "type = %d or w_type = %d is not an OB_TYPE", type, w_type);
  if (!((float)eps > 0.0f) || !std::isfinite((float)eps))
    return failf(OB_ERR_INVALID, "eps = %g must be positive", eps);
  if (sum && !residual) return failf(OB_ERR_INVALID, "sum is given without a residual");
  if (sum && sum == y) return failf(OB_ERR_INVALID, "y and sum are the same array");
  OB_TRY(check_sizes(rows, cols));
  if (rows == 0 || cols == 0) return OB_OK;
  OB_TRY(check_rows(x, ldx, rows, cols, type, "x"));
  OB_TRY(check_rows(y, ldy, rows, cols, type, "y"));
  if (residual) OB_TRY(check_rows(residual, ldr, rows, cols, type, "residual"));
  if (sum) OB_TRY(check_rows(sum, lds, rows, cols, type, "sum"));
  if (weight) OB_TRY(check_ptr(weight, type_bytes(w_type), "weight"));
  if (bias) OB_TRY(check_ptr(bias, type_bytes(w_type), "bias"));
  if (mean) OB_TRY(check_ptr(mean, 4, "mean"));
  if (rstd) OB_TRY(check_ptr(rstd, 4, "rstd"));
  ob::LayerNormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.sum = sum;
  a.mean = mean;
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.lds = lds;
  a.rows = rows;
  a.cols = (int)cols;
  a.w_type = w_type;
  a.eps = (float)eps;
  return launched(ob::launch_layernorm_fwd(a, type, reinterpret_cast<cudaStream_t>(stream)),
                  "layernorm_fwd");
}

ob_status ob_layernorm_workspace_bytes(size_t rows, size_t cols, size_t* bytes) {
  OB_TRACE();
  if (!bytes) return failf(OB_ERR_INVALID, "bytes is NULL");
  OB_TRY(check_sizes(rows, cols));
  *bytes = rows && cols ? layernorm_partials(rows, cols) : 0;
  return OB_OK;
}

ob_status ob_layernorm_bwd(const void* dy, size_t lddy, const void* x, size_t ldx,
                           const float* mean, const float* rstd, const void* weight, int w_type,
                           const void* dsum, size_t ldds, void* dx, size_t lddx, void* dweight,
                           void* dbias, size_t rows, size_t cols, int type, void* workspace,
                           size_t workspace_bytes, ob_stream_t stream) {
  OB_TRACE();
  if (!known_type(type) || !known_type(w_type))
    return failf(OB_ERR_INVALID, "type = %d or w_type = %d is not an OB_TYPE", type, w_type);
  OB_TRY(check_sizes(rows, cols));
  if (cols == 0) return OB_OK;
  if (dweight) OB_TRY(check_ptr(dweight, type_bytes(w_type), "dweight"));
  if (dbias) OB_TRY(check_ptr(dbias, type_bytes(w_type), "dbias"));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) {
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, cols * type_bytes(w_type), s);
    if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, cols * type_bytes(w_type), s);
    return launched(e, "layernorm_bwd");
  }
  OB_TRY(check_rows(dy, lddy, rows, cols, type, "dy"));
  OB_TRY(check_rows(x, ldx, rows, cols, type, "x"));
  OB_TRY(check_ptr(mean, 4, "mean"));
  OB_TRY(check_ptr(rstd, 4, "rstd"));
  if (weight) OB_TRY(check_ptr(weight, type_bytes(w_type), "weight"));
  if (dsum && !dx) return failf(OB_ERR_INVALID, "dsum is given without dx");
  if (dsum) OB_TRY(check_rows(dsum, ldds, rows, cols, type, "dsum"));
  if (dx) OB_TRY(check_rows(dx, lddx, rows, cols, type, "dx"));
  if (!dx && !dweight && !dbias) return OB_OK;
  OB_TRY(check_workspace(workspace, workspace_bytes,
                         dweight || dbias ? layernorm_partials(rows, cols) : 0, 16));
  ob::LayerNormBwdArgs a{};
  a.dy = dy;
  a.x = x;
  a.dsum = dsum;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.lddy = lddy;
  a.ldx = ldx;
  a.ldds = ldds;
  a.lddx = lddx;
  a.rows = rows;
  a.cols = (int)cols;
  a.w_type = w_type;
  a.partial = static_cast<float*>(workspace);
  a.parts = ob::layernorm_bwd_parts(rows, (int)cols);
  return launched(ob::launch_layernorm_bwd(a, type, s), "layernorm_bwd");
}

ob_status ob_linear_workspace_bytes(const ob_linear* l, int backward, size_t* bytes) {
  OB_TRACE();
  if (!bytes) return failf(OB_ERR_INVALID, "bytes is NULL");
  OB_TRY(check_linear(l));
  *bytes = ob::linear_workspace_bytes(linear_args(*l), backward != 0);
  return OB_OK;
}

ob_status ob_linear_fwd(const ob_linear* l, const ob_matrix* x, const ob_matrix* w,
                        const void* bias, const ob_matrix* residual, const ob_matrix* z,
                        const ob_matrix* y, void* workspace, size_t workspace_bytes,
                        ob_stream_t stream) {
  OB_TRACE();
  OB_TRY(check_linear(l));
  ob::LinearArgs a = linear_args(*l);
  if (a.M == 0 || a.N == 0) return OB_OK;
  OB_TRY(check_matrix(*l, x, a.M, a.K, "x", &a.x));
  OB_TRY(check_matrix(*l, w, a.w_kn ? a.K : a.N, a.w_kn ? a.N : a.K, "w", &a.w));
  OB_TRY(check_matrix(*l, y, a.M, a.N, "y", &a.y));
  if (residual) OB_TRY(check_matrix(*l, residual, a.M, a.N, "residual", &a.residual));
  if (z) OB_TRY(check_matrix(*l, z, a.M, a.N, "z", &a.z));
  if (z && z->data == y->data) return failf(OB_ERR_INVALID, "y and z are the same array");
  if (bias) OB_TRY(check_ptr(bias, 2, "bias"));
  a.bias = bias;
  OB_TRY(check_workspace(workspace, workspace_bytes, ob::linear_workspace_bytes(a, false), 256));
  a.workspace = static_cast<uint8_t*>(workspace);
  return launched(ob::launch_linear_fwd(a, reinterpret_cast<cudaStream_t>(stream)), "linear_fwd");
}

ob_status ob_linear_bwd(const ob_linear* l, const ob_matrix* dy, const ob_matrix* x,
                        const ob_matrix* w, const ob_matrix* z, const ob_matrix* dx,
                        const ob_matrix* dw, void* dbias, void* workspace,
                        size_t workspace_bytes, ob_stream_t stream) {
  OB_TRACE();
  OB_TRY(check_linear(l));
  ob::LinearArgs a = linear_args(*l);
  OB_TRY(check_matrix(*l, dy, a.M, a.N, "dy", &a.dy));
  if (a.act != OB_ACT_NONE) OB_TRY(check_matrix(*l, z, a.M, a.N, "z", &a.z));
  const int64_t wr = a.w_kn ? a.K : a.N, wc = a.w_kn ? a.N : a.K;
  if (dx && a.M > 0 && a.K > 0) {
    OB_TRY(check_matrix(*l, w, wr, wc, "w", &a.w));
    OB_TRY(check_matrix(*l, dx, a.M, a.K, "dx", &a.dx));
  }
  if (dw && a.N > 0 && a.K > 0) {
    OB_TRY(check_matrix(*l, x, a.M, a.K, "x", &a.x));
    OB_TRY(check_matrix(*l, dw, wr, wc, "dw", &a.dw));
  }
  if (dbias && a.N > 0) {
    OB_TRY(check_ptr(dbias, 2, "dbias"));
    a.dbias = dbias;
  }
  if (!a.dx.data && !a.dw.data && !a.dbias) return OB_OK;
  OB_TRY(check_workspace(workspace, workspace_bytes, ob::linear_workspace_bytes(a, true), 256));
  a.workspace = static_cast<uint8_t*>(workspace);
  return launched(ob::launch_linear_bwd(a, reinterpret_cast<cudaStream_t>(stream)), "linear_bwd");
}

ob_status ob_layer_device_error(unsigned* code, ob_stream_t stream) {
  OB_TRACE();
  if (!code) return failf(OB_ERR_INVALID, "layer_device_error: code is NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned* words[2] = {nullptr, nullptr};
  unsigned v[2] = {0, 0};
  cudaError_t e = ob::linear_error_word(&words[0]);
  if (e == cudaSuccess) e = ob::layernorm_error_word(&words[1]);
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    e = cudaMemcpyAsync(&v[i], words[i], sizeof v[i], cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(words[i], 0, sizeof v[i], s);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return launched(e, "layer_device_error");
  *code = v[0] ? v[0] : v[1];
  return OB_OK;
}

ob_status ob_adamw_step(const ob_adamw* a, const ob_adamw_tensor* tensors,
                        const void* const* grads, int count, void* m, void* v, uint8_t* m_exp,
                        uint8_t* v_exp, double* counter, ob_stream_t stream) {
  OB_TRACE();
  if (!a) return failf(OB_ERR_INVALID, "adamw is NULL");
  if (a->state_bits != 8 && a->state_bits != 32)
    return failf(OB_ERR_INVALID, "state_bits = %d must be 8 or 32", a->state_bits);
  if (!known_type(a->grad_type))
    return failf(OB_ERR_INVALID, "grad_type = %d is not an OB_TYPE", a->grad_type);
  if (!(a->lr >= 0.0) || !std::isfinite(a->lr))
    return failf(OB_ERR_INVALID, "lr = %g must not be negative", a->lr);
  if (!(a->b1 >= 0.0 && a->b1 < 1.0 && a->b2 >= 0.0 && a->b2 < 1.0))
    return failf(OB_ERR_INVALID, "b1 = %g, b2 = %g must be in [0, 1)", a->b1, a->b2);
  if (!(a->eps >= 1e-12 && a->eps <= 1.0))
    return failf(OB_ERR_INVALID, "eps = %g must be in [1e-12, 1]", a->eps);
  if (count < 0) return failf(OB_ERR_INVALID, "count = %d is negative", count);
  if (count && (!tensors || !grads)) return failf(OB_ERR_INVALID, "tensors or grads is NULL");
  OB_TRY(check_ptr(counter, 8, "counter"));
  if (a->lr_device) OB_TRY(check_ptr(a->lr_device, 4, "lr_device"));
  if (a->grad_scale) OB_TRY(check_ptr(a->grad_scale, 4, "grad_scale"));
  if (a->skip) OB_TRY(check_ptr(a->skip, 4, "skip"));
  std::vector<ob::AdamTensor> list;
  try {
    list.resize(count);
  } catch (const std::bad_alloc&) {
    return failf(OB_ERR_INVALID, "no memory for %d tensors", count);
  }
  uint64_t blocks = 0;
  for (int i = 0; i < count; ++i) {
    const ob_adamw_tensor& t = tensors[i];
    if (!known_type(t.p_type) || (t.copy && !known_type(t.copy_type)))
      return failf(OB_ERR_INVALID, "tensor %d: a type is not an OB_TYPE", i);
    if (!(t.decay >= 0.0f) || !std::isfinite(t.decay))
      return failf(OB_ERR_INVALID, "tensor %d: decay = %g must not be negative", i,
                   (double)t.decay);
    if (t.n > (1ull << 40)) return failf(OB_ERR_INVALID, "tensor %d is over 2^40 elements", i);
    auto lies = [](const void* p, int type) { return reinterpret_cast<uintptr_t>(p) % type_bytes(type) == 0; };
    if (t.n && !t.p) return failf(OB_ERR_INVALID, "tensor %d: p is NULL", i);
    if (t.n && !(lies(t.p, t.p_type) && (!t.copy || lies(t.copy, t.copy_type)) && lies(grads[i], a->grad_type)))
      return failf(OB_ERR_ALIGN, "tensor %d: p, copy or gradient is not aligned to its element", i);
    list[i] = ob::AdamTensor{t.p, grads[i], t.copy, t.n, blocks, t.decay,
                             t.p_type | (t.copy ? t.copy_type : 0) << 8};
    blocks += (t.n + ob::kAdamBlock - 1) / ob::kAdamBlock;
    if (blocks > (1ull << 32))
      return failf(OB_ERR_INVALID, "the tensors are over 2^40 elements");
  }
  if (blocks) {
    OB_TRY(check_ptr(m, 32, "m"));
    OB_TRY(check_ptr(v, 32, "v"));
    if (a->state_bits == 8) {
      OB_TRY(check_ptr(m_exp, 1, "m_exp"));
      OB_TRY(check_ptr(v_exp, 1, "v_exp"));
    }
  }
  ob::AdamArgs r{};
  r.bits = a->state_bits;
  r.g_type = a->grad_type;
  r.lr = a->lr;
  r.b1 = a->b1;
  r.b2 = a->b2;
  r.eps = (float)a->eps;
  r.seed = a->seed;
  r.lr_device = a->lr_device;
  r.grad_scale = a->grad_scale;
  r.skip = a->skip;
  r.m = m;
  r.v = v;
  r.m_exp = m_exp;
  r.v_exp = v_exp;
  r.counter = counter;
  return launched(ob::launch_adamw(r, list.data(), count, reinterpret_cast<cudaStream_t>(stream)),
                  "adamw_step");
}

ob_status ob_adamw_moments(const void* m, const void* v, const uint8_t* m_exp,
                           const uint8_t* v_exp, size_t elements, void* m_out, void* v_out,
                           ob_stream_t stream) {
  OB_TRACE();
  if (elements % ob::kAdamBlock || elements > (1ull << 40))
    return failf(OB_ERR_INVALID, "elements = %zu must be a multiple of 256, at most 2^40",
                 elements);
  if (elements == 0) return OB_OK;
  OB_TRY(check_ptr(m, 16, "m"));
  OB_TRY(check_ptr(v, 16, "v"));
  OB_TRY(check_ptr(m_exp, 1, "m_exp"));
  OB_TRY(check_ptr(v_exp, 1, "v_exp"));
  OB_TRY(check_ptr(m_out, 16, "m_out"));
  OB_TRY(check_ptr(v_out, 16, "v_out"));
  return launched(
      ob::launch_adamw_moments(static_cast<const uint8_t*>(m), static_cast<const uint8_t*>(v),
                               m_exp, v_exp, elements, m_out, v_out,
                               reinterpret_cast<cudaStream_t>(stream)),
      "adamw_moments");
}

}  // extern "C"
