// A mixture-of-experts layer for a few tokens: router and top-k, the gated
// products of the chosen experts, and their weighted sum.
#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "moe.cuh"

namespace effort {

// One block per token: the logits by warps, then the top-k by one thread.
__global__ void __launch_bounds__(256) k_moe_router(MoeCall c) {
  __shared__ float logit[EFFORT_MAX_EXPERTS];
  const int t = blockIdx.x, lane = threadIdx.x & 31, E = c.n_experts;
  for (int e = threadIdx.x >> 5; e < E; e += 8) {
    float s = 0.0f;
    for (int k = lane; k < c.I; k += 32)
      s += load_dt(c.x, c.xdt, t * c.xstride + k) * load_dt(c.router, c.rdt, (size_t)e * c.I + k);
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
    if (lane == 0) logit[e] = s;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  const float nan = __int_as_float(0x7fffffff);
  bool bad = false;
  float top = -INFINITY, all = 0.0f, sum = 0.0f;
  for (int e = 0; e < E; ++e) {
    bad |= logit[e] != logit[e];
    top = fmaxf(top, logit[e]);
  }
  for (int e = 0; e < E; ++e) all += expf(logit[e] - top);
  unsigned long long used[EFFORT_MAX_EXPERTS / 64] = {};
  for (int j = 0; j < c.top_k; ++j) {
    int best = -1;
    for (int e = 0; e < E; ++e) {
      if (used[e / 64] >> (e % 64) & 1) continue;
      const float l = logit[e] == logit[e] ? logit[e] : -INFINITY;
      if (best < 0 || l > (logit[best] == logit[best] ? logit[best] : -INFINITY)) best = e;
    }
    used[best / 64] |= 1ull << (best % 64);
    const float g = expf(logit[best] - top);
    sum += g;
    c.ids[t * c.top_k + j] = best;
    c.gates[t * c.top_k + j] = g;
  }
  const float d = c.gate_mode == EFFORT_GATE_SOFTMAX_OF_TOP ? sum : all;
  for (int j = 0; j < c.top_k; ++j)
    c.gates[t * c.top_k + j] = bad ? nan : __fdiv_rn(c.gates[t * c.top_k + j], d);
}

__device__ __forceinline__ float weight_at(const uint8_t* core, int wk, int r, int k) {
  if (wk == kWE4M3) return e4m3_to_float(core[core_offset(r, k, 1)]);
  const void* p = core + core_offset(r, k, 2);
  return wk == kWF16 ? __half2float(*(const __half*)p) : __bfloat162float(*(const __nv_bfloat16*)p);
}

// One warp per (pair, hidden unit): both dot products, then silu(a) b.
__global__ void __launch_bounds__(256) k_moe_up(MoeCall c) {
  const int lane = threadIdx.x & 31, p = blockIdx.y, j = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int e = c.ids[p];
  if (j >= c.F || e < 0 || e >= c.n_experts) return;
  const int t = p / c.top_k, ke = k_per_block(c.wk);
  const uint8_t* base = c.w13.data + e * c.w13.stride;
  float a = 0.0f, b = 0.0f;
  for (int kb = 0; kb < c.w13.nkb; ++kb) {
    const uint8_t* c1 = base + core_at(2 * (j / 8), kb, c.w13.nkb);
    const uint8_t* c3 = base + core_at(2 * (j / 8) + 1, kb, c.w13.nkb);
    float da = 0.0f, db = 0.0f;
    for (int k = lane; k < ke; k += 32) {
      const int kk = kb * ke + k;
      if (kk >= c.I) break;
      const float x = load_dt(c.x, c.xdt, t * c.xstride + kk);
      da += x * weight_at(c1, c.wk, j % 8, k);
      db += x * weight_at(c3, c.wk, j % 8, k);
    }
    if (c.wk == kWE4M3) {
      const size_t s = ((size_t)e * c.w13.nkb + kb) * c.nsb13 + j / kBlk;
      da *= c.s1[s];
      db *= c.s3[s];
    }
    a += da;
    b += db;
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) {
    a += __shfl_xor_sync(~0u, a, m);
    b += __shfl_xor_sync(~0u, b, m);
  }
  if (lane == 0) c.h[(size_t)p * c.hstride + j] = a / (1.0f + expf(-a)) * b;
}

// One warp per (token, output): the products of all its pairs.
__global__ void __launch_bounds__(256) k_moe_down(MoeCall c) {
  const int lane = threadIdx.x & 31, t = blockIdx.y, i = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= c.I) return;
  const int ke = k_per_block(c.wk);
  float y = 0.0f;
  for (int j = 0; j < c.top_k; ++j) {
    const int p = t * c.top_k + j, e = c.ids[p];
    if (e < 0 || e >= c.n_experts) continue;
    const uint8_t* base = c.w2.data + e * c.w2.stride;
    float a = 0.0f;
    for (int kb = 0; kb < c.w2.nkb; ++kb) {
      const uint8_t* core = base + core_at(i / 8, kb, c.w2.nkb);
      float d = 0.0f;
      for (int k = lane; k < ke; k += 32) {
        const int kk = kb * ke + k;
        if (kk >= c.F) break;
        d += c.h[(size_t)p * c.hstride + kk] * weight_at(core, c.wk, i % 8, k);
      }
      if (c.wk == kWE4M3) d *= c.s2[((size_t)e * c.w2.nkb + kb) * c.nsb2 + i / kBlk];
      a += d;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) a += __shfl_xor_sync(~0u, a, m);
    y += c.gates[p] * a;
  }
  if (lane == 0) store_dt(c.out, c.odt, t * c.ostride + i, y);
}

cudaError_t launch_moe(const MoeCall& c, cudaStream_t s) {
  if (c.gate_mode != EFFORT_GATE_GIVEN) k_moe_router<<<c.n_tokens, 256, 0, s>>>(c);
  k_moe_up<<<dim3((unsigned)cdiv(c.F, 8), (unsigned)(c.n_tokens * c.top_k)), 256, 0, s>>>(c);
  k_moe_down<<<dim3((unsigned)cdiv(c.I, 8), (unsigned)c.n_tokens), 256, 0, s>>>(c);
  return cudaGetLastError();
}

// hidden activations of every pair, fp32
size_t moe_scratch_bytes(int n_tokens, int top_k, int F, int wk) {
  const int ke = k_per_block(wk);
  return (size_t)n_tokens * top_k * cdiv(F, ke) * ke * 4;
}

}  // namespace effort
