// What one mixture-of-experts call hands to its kernels.
#pragma once
#include "ffn_common.cuh"

namespace effort {

struct MoeCall {
  TileMat w13, w2;              // cores of w1 and w3 in turn; w2
  const float *s1, *s3, *s2;    // e4m3: scales [expert][K block][128 rows]
  int nsb13, nsb2;              // their row blocks
  const void* router;
  int rdt, wk, n_experts, I, F;
  const void* x;
  int xdt;
  long long xstride;
  int n_tokens, top_k, gate_mode;
  int* ids;
  float* gates;
  void* out;
  int odt;
  long long ostride;
  float* h;                     // [pairs][hstride] hidden activations
  long long hstride;
};

}  // namespace effort
