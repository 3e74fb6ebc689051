// Argument blocks and launchers of the operators of a layer (layer norm, the
// dense layer's products) and of the AdamW step over many tensors.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "ob.h"

namespace ob {

struct LayerNormArgs {
  const void *x, *residual;      // residual or null
  const void *weight, *bias;     // or null
  void *y, *sum;                 // sum or null
  float *mean, *rstd;            // or null (forward)
  uint64_t ldx, ldr, ldy, lds;
  uint64_t rows;
  int cols, w_type;
  float eps;
};

struct LayerNormBwdArgs {
  const void *dy, *x, *dsum;     // dsum or null
  const void* weight;            // or null
  const float *mean, *rstd;
  void *dx, *dweight, *dbias;    // each or null
  uint64_t lddy, ldx, ldds, lddx;
  uint64_t rows;
  int cols, w_type;
  float* partial;                // [parts][2][cols]
  int parts;
};

cudaError_t launch_layernorm_fwd(const LayerNormArgs& a, int type, cudaStream_t s);
// Blocks whose partial sums the gradient of these sizes keeps.
int layernorm_bwd_parts(uint64_t rows, int cols);
cudaError_t launch_layernorm_bwd(const LayerNormBwdArgs& a, int type, cudaStream_t s);

// A matrix of 16-bit elements: element (i, j) at data + i * ld + j.
struct Mat {
  void* data;
  int64_t ld;
};

// A map of `rows` rows of `cols` elements whose boxes are box_rows rows of 64 or 32
// elements, swizzled as far as they are wide; what is outside reads as zero.
cudaError_t matrix_tensor_map(CUtensorMap* map, const Mat& m, int type, int64_t rows, int64_t cols,
                              int box_cols, int box_rows);

struct LinearArgs {
  int type, act, w_kn, unaligned;
  int64_t M, N, K;
  Mat x, w, y, z, residual;      // z and residual: data or null
  const void* bias;              // or null
  Mat dy, dx, dw;                // backward; dx and dw: data or null
  void* dbias;                   // or null
  uint8_t* workspace;
};

size_t linear_workspace_bytes(const LinearArgs& a, bool backward);
cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_bwd(const LinearArgs& a, cudaStream_t s);
// The device words where a wait that ran out leaves its code.
cudaError_t linear_error_word(unsigned** word);
cudaError_t layernorm_error_word(unsigned** word);

// ---------------------------------------------------------------------------
// One product C[M][N] = sum over k of A(m, k) B(n, k) with the dense layer's
// epilogue (k_gemm.cu).
// ---------------------------------------------------------------------------

struct Epilogue {
  const void* bias;          // [N], or null
  Mat residual, z, out;      // residual and z: data or null
  int act, type;
  int tiled;                 // every matrix, and bias, lies on 16 bytes
};

struct Gemm {
  Mat a, b;
  int a_mn, b_mn;            // stored [K][M] or [K][N] instead of [M][K] or [N][K]
  int64_t M, N, K;
  int pair;                  // one of launch_gemms' two
  Epilogue ep;
  float* partial;            // gemm_partial_bytes
};

// By sizes, a_mn and pair alone.
size_t gemm_partial_bytes(int64_t M, int64_t N, int64_t K, bool a_mn, bool pair);
// Whether a product has so few rows of A, stored [M][K], that B's way through the memory
// bounds it: it has a kernel of its own (k_few.cu).
bool few_rows(int64_t M, int64_t N, int64_t K, bool a_mn, bool pair);
cudaError_t launch_few(const Gemm& g, cudaStream_t s);
cudaError_t launch_gemm(const Gemm& g, cudaStream_t s);
// Two products, in one launch where the card has room for both; their partials are apart.
cudaError_t launch_gemms(const Gemm& g, const Gemm& h, cudaStream_t s);

constexpr int kAdamBlock = 256;  // elements that share a unit, and the state's grain

struct AdamTensor {
  void* p;
  const void* g;     // null: the tensor is left as it is
  void* copy;        // or null
  uint64_t n;
  uint64_t first;    // its first block in the state
  float decay;
  int types;         // p_type | copy_type << 8; from bit 16 on, all lie on 16 (32) bytes
};

struct AdamArgs {
  int bits, g_type;
  double lr, b1, b2;
  float eps;
  uint64_t seed;
  const float *lr_device, *grad_scale, *skip;
  void *m, *v;
  uint8_t *m_exp, *v_exp;
  double* counter;
};

cudaError_t launch_adamw(const AdamArgs& a, const AdamTensor* t, int count, cudaStream_t s);
cudaError_t launch_adamw_moments(const uint8_t* m, const uint8_t* v, const uint8_t* m_exp,
                                 const uint8_t* v_exp, size_t elements, void* m_out, void* v_out,
                                 cudaStream_t s);

}  // namespace ob
