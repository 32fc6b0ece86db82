// The step between two blocks of a decoder layer: norm of the block's output,
// gate, scaled residual, norm for the next block, and its e4m3 quantisation.
//
//   u = post(y);  x' = a x + b g u;  h = pre(x');  s = max|h| over 128 / 448, q = h / s
//
// One thread block per row, the row held in shared memory in fp32 between the
// passes, so every input is read once and every output written once.
#include "../../include/effort.h"
#include "ffn_common.cuh"

namespace effort {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  float t = 0.0f;
  for (int w = 0; w < nw; ++w) t += red[w];
  return t;
}

// (v - mean) / sqrt(mean((v - mean)^2) + eps) * (off + w) + b over a row in shared memory
__device__ void norm_row(float* row, int n, int kind, const void* w, const void* b, int wdt, float off, float eps,
                         float* red) {
  float mean = 0.0f;
  if (kind == EFFORT_NORM_LAYER) {
    float s = 0.0f;
    for (int i = threadIdx.x; i < n; i += blockDim.x) s += row[i];
    mean = block_sum(s, red) / (float)n;
  }
  float q = 0.0f;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const float d = row[i] - mean;
    q += d * d;
  }
  const float r = rsqrtf(block_sum(q, red) / (float)n + eps);
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    float v = (row[i] - mean) * r;
    if (w) v *= off + load_dt(w, wdt, i);
    if (b) v += load_dt(b, wdt, i);
    row[i] = v;
  }
}

__global__ void __launch_bounds__(kNormThreads) k_block_norm(effort_block_norm_t a) {
  extern __shared__ float row[];
  __shared__ float red[32];
  const int n = (int)a.dim;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    if (a.y) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) row[i] = load_dt(a.y, a.dtype, r * a.y_stride + i);
      if (a.post_kind != EFFORT_NORM_NONE)
        norm_row(row, n, a.post_kind, a.post_weight, a.post_bias, a.weight_dtype, a.weight_offset, a.eps, red);
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        float u = row[i];
        if (a.gate) u *= load_dt(a.gate, a.dtype, r * a.gate_stride + i);
        row[i] = a.residual_scale * load_dt(a.x, a.dtype, r * a.x_stride + i) + a.branch_scale * u;
      }
    } else {
      for (int i = threadIdx.x; i < n; i += blockDim.x)
        row[i] = a.residual_scale * load_dt(a.x, a.dtype, r * a.x_stride + i);
    }
    if (a.x_out)
      for (int i = threadIdx.x; i < n; i += blockDim.x) store_dt(a.x_out, a.dtype, r * a.x_out_stride + i, row[i]);
    if (a.pre_kind != EFFORT_NORM_NONE)
      norm_row(row, n, a.pre_kind, a.pre_weight, a.pre_bias, a.weight_dtype, a.weight_offset, a.eps, red);
    if (a.h_out)
      for (int i = threadIdx.x; i < n; i += blockDim.x) store_dt(a.h_out, a.h_dtype, r * a.h_stride + i, row[i]);
    if (a.q_out) {
      __syncthreads();
      const int lane = threadIdx.x & 31;
      for (int b = threadIdx.x >> 5; b * kBlk < n; b += kNormThreads / 32) {
        float v[4], m = 0.0f;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = b * kBlk + 32 * j + lane;
          v[j] = i < n ? row[i] : 0.0f;
          m = fmaxf(m, fabsf(v[j]));
          nan |= v[j] != v[j];
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
        const float s = __any_sync(~0u, nan) ? __int_as_float(0x7fffffff) : __fdiv_rn(m, kE4M3Max);
        if (lane == 0) a.q_scales[r * a.q_scales_stride + b] = s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = b * kBlk + 32 * j + lane;
          if (i < n)
            static_cast<uint8_t*>(a.q_out)[r * a.q_stride + i] =
                (uint8_t)__nv_cvt_float_to_fp8(s == 0.0f ? 0.0f : __fdiv_rn(v[j], s), __NV_SATFINITE, __NV_E4M3);
        }
      }
    }
    __syncthreads();  // the row is free for the next one
  }
}

cudaError_t launch_block_norm(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  const size_t smem = (size_t)a.dim * 4;
  cudaError_t e = cudaFuncSetAttribute(k_block_norm, cudaFuncAttributeMaxDynamicSharedMemorySize, EFFORT_MAX_IN_DIM * 4);
  if (e != cudaSuccess) return e;
  const long long grid = a.rows < 8ll * sms ? a.rows : 8ll * sms;
  k_block_norm<<<(unsigned)grid, kNormThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace effort
