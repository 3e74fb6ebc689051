// Argument block and launchers of the attention.
#pragma once

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

}  // namespace ob
