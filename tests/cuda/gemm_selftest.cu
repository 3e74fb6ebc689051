// Test-only entry to the dense layer's product (csrc/k_gemm.cu) with `lost` bytes a step that
// its barriers count and no copy brings: its waits have to run out, leave their code, let what
// is in flight land and let the kernel end.  Built by tests/test_gpu_gemm_waits.py with nvcc
// into a temporary shared library.
#include "k_gemm.cu"

namespace {

template <int CG>
cudaError_t product(const ob::Gemm& g, const ob::Plan& p, uint32_t lost) {
  ob::GemmArgs a{};
  cudaError_t e = ob::fill<CG>(g, p, &a);
  a.stage += lost;
  if (e == cudaSuccess) e = ob::run_products<CG>(a, a.workers * CG, nullptr);
  return e == cudaSuccess ? cudaDeviceSynchronize() : e;
}

}  // namespace

// y [M][N] = x [M][K] w [N][K]^T + residual in bf16, every array contiguous and on 16 bytes, by
// blocks (pairs 0) or pairs of blocks on whole tiles; *code gets the error word, which is cleared.
extern "C" int gemm_selftest(void* x, void* w, void* residual, void* y, long long M, long long N,
                             long long K, int pairs, unsigned lost, unsigned* code) {
  ob::Gemm g{};
  g.a = {x, K};
  g.b = {w, K};
  g.M = M;
  g.N = N;
  g.K = K;
  g.ep.residual = {residual, N};
  g.ep.out = {y, N};
  g.ep.type = OB_TYPE_BF16;
  g.ep.tiled = 1;
  const int edge = pairs ? 256 : 128;
  ob::Plan p{};
  p.cg = pairs ? 2 : 1;
  p.tiles_m = (int)((M + edge - 1) / edge);
  p.tiles_n = (int)((N + edge - 1) / edge);
  p.steps = (int)((K + ob::BK - 1) / ob::BK);
  p.whole = p.tiles_m * p.tiles_n;
  p.workers = p.whole < ob::kSms / p.cg ? p.whole : ob::kSms / p.cg;
  cudaError_t e = pairs ? product<2>(g, p, lost) : product<1>(g, p, lost);
  unsigned* word = nullptr;
  if (e == cudaSuccess) e = ob::linear_error_word(&word);
  if (e == cudaSuccess) e = cudaMemcpy(code, word, sizeof *code, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(word, 0, sizeof *code);
  return (int)e;
}
