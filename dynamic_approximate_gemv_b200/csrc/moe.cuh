// What one mixture-of-experts call hands to its kernels.
#pragma once
#include "stream.cuh"

namespace effort {

struct MoeCall {
  TileMat w13, w2;              // cores of w1 and w3 in turn; w2
  const float *s1, *s3, *s2;    // e4m3: scales [expert][row block][align4(K blocks)]
  int nsb13, nsb2;              // their row blocks
  const void* router;           // [expert][rpitch], rows padded with zeros
  int rdt, rpitch, wk, n_experts, I, F;
  const void* x;
  int xdt;
  long long xstride;
  int n_tokens, top_k, gate_mode;
  int* ids;
  float* gates;
  void* out;
  int odt;
  long long ostride;
  bool spread;                  // column norms of w1 or w3 differ much within some K block
  const double2* bound;         // [expert][hidden K block] largest column norms of w1 and w3
  // scratch
  char* xop;                    // [tokens] rows of activation blocks (stream.cuh)
  double* xnorm;                // [tokens] their norms
  char* h;                      // [pairs] hidden activations, likewise
  float* z;                     // [K share][pairs][I] second products
  int xpitch, hpitch, shares;   // bytes of a row; parts of the second product's K
  WaitHook hook;
};

// scratch of a call in bytes, carved into c where c is given (base: the caller's memory)
size_t moe_scratch(MoeCall* c, char* base, int n_tokens, int top_k, int n_experts, int I, int F, int wk, int nkb13,
                   int nkb2, int sms);

}  // namespace effort
