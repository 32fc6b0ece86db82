// The product with e4m3 operands and one scale for each block of 128:
//
//   out[r][n] = sum_b xs[r][b] ws[b][n / 128] sum_{k in b} x[r][k] w[k][n]
//
// and the layout of its weights.
#include "../../include/effort.h"
#include "ffn_common.cuh"

namespace effort {

// [K x N] row-major (K = in, N = out) into cores.  One block of 256 threads
// per (matrix, K block, 64 columns); columns col0 + c become row
// map(col0 + c) of the stored matrix: with pair = 0 the row is the column,
// with pair = 1 or 2 the cores of two matrices alternate (a layer's w1 and
// w3: core 2 j holds w1's columns 8 j .. 8 j + 7, core 2 j + 1 w3's).
template <typename T>
__global__ void __launch_bounds__(256) k_tile_weights(const T* __restrict__ w, int K, int N, uint8_t* out, int cores,
                                                      int nkb, size_t stride, int pair, unsigned* status) {
  constexpr int kKE = 128 / sizeof(T);
  __shared__ T t[kKE][64 + 16 / sizeof(T)];
  const int kb = blockIdx.x, col0 = blockIdx.y * 64, mat = blockIdx.z;
  const T* src = w + (size_t)mat * K * N;
  for (int i = threadIdx.x; i < kKE * 64; i += 256) {
    const int k = kb * kKE + i / 64, c = col0 + i % 64;
    T v = {};
    if (k < K && c < N) v = src[(size_t)k * N + c];
    if constexpr (sizeof(T) == 1) {
      if ((v & 0x7f) == 0x7f) atomicOr(status, 1u);
    }
    t[i / 64][i % 64] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {  // one 16-byte chunk each
    const int c = i / 8, ch = i % 8, col = col0 + c;
    const int core = pair ? 2 * (col / 8) + pair - 1 : col / 8;
    if (core >= cores) continue;
    alignas(16) T v[16 / sizeof(T)];
#pragma unroll
    for (int j = 0; j < (int)(16 / sizeof(T)); ++j) v[j] = t[ch * (16 / sizeof(T)) + j][c];
    const int r = col % 8;
    *reinterpret_cast<uint4*>(out + mat * stride + ((size_t)core * nkb + kb) * kCoreBytes + r * 128 + ((ch ^ r) << 4)) =
        *reinterpret_cast<const uint4*>(v);
  }
}

// 16-bit values of any kind that are inf or NaN: all exponent bits set
__global__ void k_check_finite16(const uint16_t* p, size_t n, unsigned mask, unsigned* status) {
  bool bad = false;
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
    bad |= (p[i] & mask) == mask;
  if (bad) atomicOr(status, 1u);
}
__global__ void k_check_finite32(const float* p, size_t n, unsigned* status) {
  bool bad = false;
  for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
    bad |= !isfinite(p[i]);
  if (bad) atomicOr(status, 1u);
}

cudaError_t launch_tile_weights(int wk, const void* w, int mats, int K, int N, uint8_t* out, int cores, int nkb,
                                size_t stride, int pair, unsigned* status, cudaStream_t s) {
  // enough column groups to write every core, the padded ones too
  const int cols = pair ? cores / 2 * 8 : cores * 8;
  const dim3 grid((unsigned)nkb, (unsigned)cdiv(cols, 64), (unsigned)mats);
  if (wk == kWE4M3) {
    k_tile_weights<uint8_t><<<grid, 256, 0, s>>>((const uint8_t*)w, K, N, out, cores, nkb, stride, pair, status);
  } else {
    k_tile_weights<uint16_t><<<grid, 256, 0, s>>>((const uint16_t*)w, K, N, out, cores, nkb, stride, pair, status);
    k_check_finite16<<<1024, 256, 0, s>>>((const uint16_t*)w, (size_t)mats * K * N, wk == kWF16 ? 0x7c00u : 0x7f80u,
                                          status);
  }
  return cudaGetLastError();
}
cudaError_t launch_check_finite(const float* p, size_t n, unsigned* status, cudaStream_t s) {
  k_check_finite32<<<256, 256, 0, s>>>(p, n, status);
  return cudaGetLastError();
}

// One warp per (row, 8 output columns): lane l multiplies the 4 values 4 l ..
// 4 l + 3 of each K block.
__global__ void __launch_bounds__(256) k_fp8_rows(TileMat w, const float* __restrict__ ws, int nsb, int I, int O,
                                                  const uint8_t* __restrict__ x, long long xstride,
                                                  const float* __restrict__ xs, long long xsstride, long long rows,
                                                  int odt, void* out, long long ostride) {
  const int lane = threadIdx.x & 31;
  const long long ncores = cdiv(O, 8);
  const long long unit = blockIdx.x * 8ll + (threadIdx.x >> 5);
  if (unit >= rows * ncores) return;
  const long long r = unit / ncores;
  const int core = (int)(unit % ncores);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int kb = 0; kb < w.nkb; ++kb) {
    float xv[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int k = kb * kBlk + 4 * lane + m;
      xv[m] = k < I ? e4m3_to_float(x[r * xstride + k]) : 0.0f;
    }
    const float s = xs[r * xsstride + kb] * ws[(size_t)kb * nsb + core / 16];
    const uint8_t* c = w.data + ((size_t)core * w.nkb + kb) * kCoreBytes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = *reinterpret_cast<const uint32_t*>(c + core_offset(j, 4 * lane, 1));
      float d = 0.0f;
#pragma unroll
      for (int m = 0; m < 4; ++m) d += xv[m] * e4m3_to_float((uint8_t)(b >> (8 * m)));
      acc[j] += d * s;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int m = 16; m; m >>= 1) acc[j] += __shfl_xor_sync(~0u, acc[j], m);
    if (lane == j && core * 8 + j < O) store_dt(out, odt, r * ostride + core * 8 + j, acc[j]);
  }
}

cudaError_t launch_fp8_matmul(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                              const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                              cudaStream_t s) {
  const long long blocks = (rows * cdiv(O, 8) + 7) / 8;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  k_fp8_rows<<<(unsigned)blocks, 256, 0, s>>>(w, ws, cdiv(O, kBlk), I, O, x, xstride, xs, xsstride, rows, odt, out,
                                              ostride);
  return cudaGetLastError();
}

}  // namespace effort
