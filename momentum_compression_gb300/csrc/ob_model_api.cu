// C entry points of the model-side operators (declared in ob.h): dropout,
// the relative position bias by buckets with its gradient, and the attention
// that uses both.  Arguments are checked on the host before any CUDA call.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "attn.cuh"
#include "model.cuh"
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

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_type(int t) { return t == OB_TYPE_F32 || t == OB_TYPE_BF16 || t == OB_TYPE_F16; }
size_t type_bytes(int t) { return t == OB_TYPE_F32 ? 4 : 2; }

#define OB_MODEL_PTR(ptr, al, name)                                                       \
  do {                                                                                    \
    if (!(ptr)) return failf(OB_ERR_INVALID, "%s is NULL", name);                         \
    if (!aligned((ptr), (al)))                                                            \
      return failf(OB_ERR_ALIGN, "%s is not %d-byte aligned", name, (int)(al));           \
  } while (0)

constexpr int64_t kMaxLen = 1ll << 30;
constexpr int kMaxDistance = 1 << 20;

// A natural number in 32-bit limbs, least significant first: just what the
// exact bucket edges need.
struct Natural {
  uint32_t limb[160];
  int n;
  explicit Natural(uint32_t x) : n(1) { limb[0] = x; }
  void times(uint32_t x) {
    uint64_t carry = 0;
    for (int i = 0; i < n; ++i) {
      carry += (uint64_t)limb[i] * x;
      limb[i] = (uint32_t)carry;
      carry >>= 32;
    }
    if (carry) limb[n++] = (uint32_t)carry;
  }
  bool less(const Natural& o) const {
    if (n != o.n) return n < o.n;
    for (int i = n - 1; i >= 0; --i)
      if (limb[i] != o.limb[i]) return limb[i] < o.limb[i];
    return false;
  }
};

// x^a * y^b.  a + b <= 64 factors (a side has at most 128 buckets, half of
// them logarithmic) of at most 21 bits: 42 limbs.
Natural power_product(uint32_t x, int a, uint32_t y, int b) {
  Natural r(1);
  for (int i = 0; i < a; ++i) r.times(x);
  for (int i = 0; i < b; ++i) r.times(y);
  return r;
}

ob_status check_relpos(const ob_relpos* rp) {
  if (!rp) return failf(OB_ERR_INVALID, "relpos is NULL");
  const int side = rp->two_sided ? rp->num_buckets / 2 : rp->num_buckets;
  bool ok = rp->side == side && side >= 2 && side <= OB_RELPOS_MAX_SIDE &&
            rp->num_buckets == (rp->two_sided ? 2 * side : side);
  // The edges index shared memory: as ob_relpos_init leaves them, and none else.
  for (int b = 0; ok && b < side; ++b)
    ok = b < side / 2 ? rp->first[b] == b
                      : rp->first[b] >= rp->first[b - 1] && rp->first[b] <= kMaxDistance;
  if (!ok) return failf(OB_ERR_INVALID, "relpos is not one that ob_relpos_init filled");
  return OB_OK;
}

ob_status check_lengths(int64_t Lq, int64_t Lk, int64_t q_offset, int64_t most) {
  if (Lq < 0 || Lk < 0 || Lq >= most || Lk >= most)
    return failf(OB_ERR_INVALID, "Lq = %lld, Lk = %lld must be in [0, %lld)", (long long)Lq,
                 (long long)Lk, (long long)most);
  if (q_offset <= -most || q_offset >= most)
    return failf(OB_ERR_INVALID, "q_offset = %lld is out of range", (long long)q_offset);
  return OB_OK;
}

size_t relpos_partial_bytes(const ob::RelposBwdArgs& a) {
  return (size_t)ob::relpos_bwd_blocks(a) * a.H * a.rp.num_buckets * sizeof(float);
}

// What does not depend on the arrays.
ob_status check_attn(const ob_attn* a) {
  if (!a) return failf(OB_ERR_INVALID, "attn is NULL");
  if (a->type != OB_TYPE_BF16 && a->type != OB_TYPE_F16)
    return failf(OB_ERR_UNSUPPORTED, "type = %d: attention takes OB_TYPE_BF16 and OB_TYPE_F16",
                 a->type);
  if (a->B < 0 || a->H < 1 || a->Hkv < 1 || a->H % a->Hkv || (int64_t)a->B * a->H > 65535)
    return failf(OB_ERR_INVALID,
                 "B = %d, H = %d, Hkv = %d: H must be a multiple of Hkv, B * H at most 65535", a->B,
                 a->H, a->Hkv);
  if (a->D < 8 || a->D > 128 || a->D % 8)
    return failf(OB_ERR_UNSUPPORTED, "D = %d must be a multiple of 8 in [8, 128]", a->D);
  if (ob_status st = check_lengths(a->Lq, a->Lk, a->q_offset, 1ll << 23)) return st;
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
    return failf(OB_ERR_INVALID, "scale = %g must be positive", (double)a->scale);
  if (!(a->p >= 0.0 && a->p <= 255.0 / 256))
    return failf(OB_ERR_INVALID, "p = %g must be in [0, 255/256]", a->p);
  if (a->relpos) {
    if (ob_status st = check_relpos(a->relpos)) return st;
    const int last = a->relpos->first[a->relpos->side - 1];
    if (last * (a->relpos->two_sided ? 2 : 1) > OB_ATTN_MAX_SPAN)
      return failf(OB_ERR_UNSUPPORTED, "a bias whose buckets span %d distances: attention takes %d",
                   last * (a->relpos->two_sided ? 2 : 1), OB_ATTN_MAX_SPAN);
    OB_MODEL_PTR(a->table, 2, "table");
  } else if (a->table) {
    return failf(OB_ERR_INVALID, "table is given without relpos");
  }
  if (a->kv_len) OB_MODEL_PTR(a->kv_len, 4, "kv_len");
  return OB_OK;
}

// One of the [B][L][n][D] arrays; where an extent is 1 its stride is not used
// and becomes a harmless one.
ob_status check_heads(const ob_attn& a, const ob_heads* t, int64_t L, int n, const char* name,
                      ob::Heads* out) {
  *out = ob::Heads{nullptr, 8, 8, 8};
  if (a.B == 0 || L == 0) return OB_OK;
  if (!t) return failf(OB_ERR_INVALID, "%s is NULL", name);
  OB_MODEL_PTR(t->data, 16, name);
  const int64_t extent[3] = {a.B, L, n}, stride[3] = {t->stride_b, t->stride_l, t->stride_h};
  int64_t* to[3] = {&out->b, &out->l, &out->h};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) continue;
    if (stride[i] % 8)
      return failf(OB_ERR_ALIGN, "%s: stride %lld is not a multiple of 8 elements", name,
                   (long long)stride[i]);
    if (stride[i] < a.D || stride[i] >= (1ll << 38))
      return failf(OB_ERR_INVALID, "%s: stride %lld must be in [D, 2^38)", name,
                   (long long)stride[i]);
    *to[i] = stride[i];
  }
  out->data = t->data;
  return OB_OK;
}

ob::AttnArgs attn_args(const ob_attn& a) {
  ob::AttnArgs r{};
  r.type = a.type;
  r.B = a.B;
  r.H = a.H;
  r.Hkv = a.Hkv;
  r.D = a.D;
  r.Lq = (int)a.Lq;
  r.Lk = (int)a.Lk;
  r.causal = a.causal ? 1 : 0;
  r.q_offset = (int)a.q_offset;
  r.scale = a.scale;
  r.biased = a.relpos != nullptr;
  if (a.relpos) r.rp = *a.relpos;
  r.table = a.table;
  r.kv_len = a.kv_len;
  r.keep = ob::make_keep(a.p, a.seed, a.offset);
  return r;
}

}  // namespace

extern "C" {

ob_status ob_dropout(const void* x, size_t ldx, const void* residual, size_t ldr, void* y,
                     size_t ldy, size_t rows, size_t cols, int type, double p, uint64_t seed,
                     uint64_t offset, ob_stream_t stream) {
  OB_TRACE();
  if (!known_type(type)) return failf(OB_ERR_INVALID, "type = %d is not an OB_TYPE", type);
  if (!(p >= 0.0 && p <= 1.0)) return failf(OB_ERR_INVALID, "p = %g must be in [0, 1]", p);
  if (rows == 0 || cols == 0) return OB_OK;
  if (cols > (1ull << 40) / rows)
    return failf(OB_ERR_INVALID, "%zu rows of %zu are over 2^40 elements", rows, cols);
  const size_t s = type_bytes(type);
  OB_MODEL_PTR(x, s, "x");
  OB_MODEL_PTR(y, s, "y");
  if (residual) OB_MODEL_PTR(residual, s, "residual");
  if (rows > 1 && (ldx < cols || ldy < cols || (residual && ldr < cols)))
    return failf(OB_ERR_INVALID, "rows of %zu elements must start at least as far apart", cols);
  ob::DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.y = y;
  a.rows = rows;
  a.cols = cols;
  a.n = (uint64_t)rows * cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  if (rows == 1 || (ldx == cols && ldy == cols && (!residual || ldr == cols))) {
    a.rows = 1;
    a.cols = a.n;
  }
  a.small = a.n < (1ull << 32);
  a.magic = a.cols > 1 ? ~0ull / a.cols + 1 : 0;  // ceil(2^64 / cols)
  a.keep = ob::make_keep(p, seed, offset);
  return launched(ob::launch_dropout(a, type, reinterpret_cast<cudaStream_t>(stream)), "dropout");
}

ob_status ob_relpos_init(int num_buckets, int max_distance, int two_sided, ob_relpos* rp) {
  OB_TRACE();
  if (!rp) return failf(OB_ERR_INVALID, "relpos is NULL");
  const int most = (two_sided ? 2 : 1) * OB_RELPOS_MAX_SIDE, least = two_sided ? 4 : 2;
  if (num_buckets < least || num_buckets > most || (two_sided && num_buckets % 2))
    return failf(OB_ERR_INVALID, "num_buckets = %d must be %sin [%d, %d]", num_buckets,
                 two_sided ? "even and " : "", least, most);
  const int side = two_sided ? num_buckets / 2 : num_buckets, E = side / 2, K = side - E;
  if (max_distance <= E || max_distance > kMaxDistance)
    return failf(OB_ERR_INVALID, "max_distance = %d must be in (%d, 2^20]", max_distance, E);
  *rp = ob_relpos{};
  rp->num_buckets = num_buckets;
  rp->max_distance = max_distance;
  rp->two_sided = two_sided ? 1 : 0;
  rp->side = side;
  for (int b = 0; b < E; ++b) rp->first[b] = b;
  // first[E + k]: the first n with n^K >= D^k E^(K - k).  The logarithm says
  // where to look; the whole numbers decide.
  for (int k = 0; k < K; ++k) {
    const Natural edge = power_product((uint32_t)max_distance, k, (uint32_t)E, K - k);
    const double guess = E * std::pow((double)max_distance / E, (double)k / K);
    int n = (int)guess - 1;
    const int from = k ? rp->first[E + k - 1] : E;
    if (n < from) n = from;
    while (n > from && !power_product((uint32_t)(n - 1), K, 1, 0).less(edge)) --n;
    while (power_product((uint32_t)n, K, 1, 0).less(edge)) ++n;
    rp->first[E + k] = n;
  }
  return OB_OK;
}

ob_status ob_relpos_bias(const ob_relpos* rp, const void* table, int table_type, int H,
                         int64_t Lq, int64_t Lk, int64_t q_offset, void* out, int out_type,
                         int64_t stride_h, int64_t stride_l, ob_stream_t stream) {
  OB_TRACE();
  if (ob_status st = check_relpos(rp)) return st;
  if (!known_type(table_type) || !known_type(out_type))
    return failf(OB_ERR_INVALID, "table_type = %d or out_type = %d is not an OB_TYPE", table_type,
                 out_type);
  if (ob_status st = check_lengths(Lq, Lk, q_offset, kMaxLen)) return st;
  if (H < 0) return failf(OB_ERR_INVALID, "H = %d is negative", H);
  if (H == 0 || Lq == 0 || Lk == 0) return OB_OK;
  OB_MODEL_PTR(table, type_bytes(table_type), "table");
  OB_MODEL_PTR(out, type_bytes(out_type), "out");
  if ((Lq > 1 && stride_l < Lk) || (H > 1 && stride_h < Lk))
    return failf(OB_ERR_INVALID, "stride_l and stride_h must be at least Lk");
  ob::RelposArgs a{};
  a.rp = *rp;
  a.table = table;
  a.table_type = table_type;
  a.H = H;
  a.Lq = Lq;
  a.Lk = Lk;
  a.q_offset = q_offset;
  a.out = out;
  a.stride_h = H > 1 ? stride_h : 0;
  a.stride_l = Lq > 1 ? stride_l : 0;
  return launched(ob::launch_relpos_bias(a, out_type, reinterpret_cast<cudaStream_t>(stream)),
                  "relpos_bias");
}

ob_status ob_relpos_workspace_bytes(const ob_relpos* rp, int64_t N, int H, int64_t Lq,
                                    int64_t Lk, size_t* bytes) {
  OB_TRACE();
  if (!bytes) return failf(OB_ERR_INVALID, "bytes is NULL");
  if (ob_status st = check_relpos(rp)) return st;
  if (ob_status st = check_lengths(Lq, Lk, 0, kMaxLen)) return st;
  if (N < 0 || N >= kMaxLen || H < 0) return failf(OB_ERR_INVALID, "N or H is out of range");
  *bytes = 0;
  if (N == 0 || H == 0 || Lq == 0 || Lk == 0) return OB_OK;
  ob::RelposBwdArgs a{};
  a.rp = *rp;
  a.N = N;
  a.H = H;
  a.Lq = Lq;
  a.Lk = Lk;
  *bytes = relpos_partial_bytes(a);
  return OB_OK;
}

ob_status ob_relpos_bias_bwd(const ob_relpos* rp, const void* dout, int out_type, int64_t N,
                             int H, int64_t Lq, int64_t Lk, int64_t stride_n, int64_t stride_h,
                             int64_t stride_l, int64_t q_offset, void* dtable, int table_type,
                             void* workspace, size_t workspace_bytes, ob_stream_t stream) {
  OB_TRACE();
  if (ob_status st = check_relpos(rp)) return st;
  if (!known_type(table_type) || !known_type(out_type))
    return failf(OB_ERR_INVALID, "table_type = %d or out_type = %d is not an OB_TYPE", table_type,
                 out_type);
  if (ob_status st = check_lengths(Lq, Lk, q_offset, kMaxLen)) return st;
  if (N < 0 || N >= kMaxLen || H < 0 || H > 65535)
    return failf(OB_ERR_INVALID, "N = %lld or H = %d is out of range", (long long)N, H);
  if (H == 0) return OB_OK;
  OB_MODEL_PTR(dtable, type_bytes(table_type), "dtable");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0 || Lq == 0 || Lk == 0)
    return launched(
        cudaMemsetAsync(dtable, 0, (size_t)rp->num_buckets * H * type_bytes(table_type), s),
        "relpos_bias_bwd");
  OB_MODEL_PTR(dout, type_bytes(out_type), "dout");
  ob::RelposBwdArgs a{};
  a.rp = *rp;
  a.dout = dout;
  a.N = N;
  a.H = H;
  a.Lq = Lq;
  a.Lk = Lk;
  a.q_offset = q_offset;
  a.stride_n = N > 1 ? stride_n : 0;
  a.stride_h = H > 1 ? stride_h : 0;
  a.stride_l = Lq > 1 ? stride_l : 0;
  a.dtable = dtable;
  a.table_type = table_type;
  if (ob::relpos_bwd_blocks(a) >= 2147483648ll)
    return failf(OB_ERR_UNSUPPORTED, "relpos_bias_bwd: too many blocks");
  OB_MODEL_PTR(workspace, 16, "workspace");
  if (workspace_bytes < relpos_partial_bytes(a))
    return failf(OB_ERR_INVALID, "workspace of %zu bytes, %zu are needed", workspace_bytes,
                 relpos_partial_bytes(a));
  a.partial = static_cast<float*>(workspace);
  return launched(ob::launch_relpos_bias_bwd(a, out_type, s), "relpos_bias_bwd");
}

ob_status ob_attn_workspace_bytes(const ob_attn* at, size_t* bytes) {
  OB_TRACE();
  if (!bytes) return failf(OB_ERR_INVALID, "bytes is NULL");
  if (ob_status st = check_attn(at)) return st;
  *bytes = ob::attn_workspace_bytes(attn_args(*at));
  return OB_OK;
}

ob_status ob_attn_fwd(const ob_attn* at, const ob_heads* q, const ob_heads* k, const ob_heads* v,
                      const ob_heads* o, float* lse, ob_stream_t stream) {
  OB_TRACE();
  if (ob_status st = check_attn(at)) return st;
  ob::AttnArgs a = attn_args(*at);
  if (a.B == 0 || a.Lq == 0) return OB_OK;
  if (ob_status st = check_heads(*at, q, at->Lq, at->H, "q", &a.q)) return st;
  if (ob_status st = check_heads(*at, k, at->Lk, at->Hkv, "k", &a.k)) return st;
  if (ob_status st = check_heads(*at, v, at->Lk, at->Hkv, "v", &a.v)) return st;
  if (ob_status st = check_heads(*at, o, at->Lq, at->H, "o", &a.o)) return st;
  if (lse) OB_MODEL_PTR(lse, 4, "lse");
  a.lse = lse;
  return launched(ob::launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)), "attn_fwd");
}

ob_status ob_attn_bwd(const ob_attn* at, const ob_heads* grad_o, const ob_heads* q,
                      const ob_heads* k, const ob_heads* v, const ob_heads* o, const float* lse,
                      const ob_heads* dq, const ob_heads* dk, const ob_heads* dv, void* dtable,
                      void* workspace, size_t workspace_bytes, ob_stream_t stream) {
  OB_TRACE();
  if (ob_status st = check_attn(at)) return st;
  ob::AttnArgs a = attn_args(*at);
  if (dtable && !at->relpos)
    return failf(OB_ERR_INVALID, "dtable is given, but there is no bias");
  if (dtable) OB_MODEL_PTR(dtable, 2, "dtable");
  a.dtable = dtable;
  if (a.B > 0 && a.Lq > 0) {
    if (ob_status st = check_heads(*at, grad_o, at->Lq, at->H, "grad_o", &a.grad_o)) return st;
    if (ob_status st = check_heads(*at, q, at->Lq, at->H, "q", &a.q)) return st;
    if (ob_status st = check_heads(*at, o, at->Lq, at->H, "o", &a.o)) return st;
    if (ob_status st = check_heads(*at, dq, at->Lq, at->H, "dq", &a.dq)) return st;
    OB_MODEL_PTR(lse, 4, "lse");
    a.lse = const_cast<float*>(lse);
  }
  if (ob_status st = check_heads(*at, k, at->Lk, at->Hkv, "k", &a.k)) return st;
  if (ob_status st = check_heads(*at, v, at->Lk, at->Hkv, "v", &a.v)) return st;
  if (ob_status st = check_heads(*at, dk, at->Lk, at->Hkv, "dk", &a.dk)) return st;
  if (ob_status st = check_heads(*at, dv, at->Lk, at->Hkv, "dv", &a.dv)) return st;
  const size_t need = ob::attn_workspace_bytes(a);
  if (need) {
    OB_MODEL_PTR(workspace, 256, "workspace");
    if (workspace_bytes < need)
      return failf(OB_ERR_INVALID, "workspace of %zu bytes, %zu are needed", workspace_bytes, need);
  }
  a.workspace = workspace;
  return launched(ob::launch_attn_bwd(a, reinterpret_cast<cudaStream_t>(stream)), "attn_bwd");
}

ob_status ob_attn_device_error(unsigned* code, ob_stream_t stream) {
  OB_TRACE();
  if (!code) return failf(OB_ERR_INVALID, "attn_device_error: code is NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned* word = nullptr;
  unsigned v = 0;
  cudaError_t e = ob::attn_error_word(&word);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof v, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof v, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return launched(e, "attn_device_error");
  *code = v;
  return OB_OK;
}

}  // extern "C"
