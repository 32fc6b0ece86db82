// The step between two blocks of a decoder layer: norm of the block's output,
// gate, scaled residual, norm for the next block, and its e4m3 quantisation.
//
//   u = post(y);  x' = a x + b g u;  h = pre(x');  s = max|h| over 128 / 448, q = h / s
//
// Bound by its bytes: every input is read once and every output written once,
// and a row stays in its block's registers in between.  One block per row,
// rows in turn; several blocks per SM, so that one row's loads run while
// another's sums are joined.  A warp owns whole blocks of 128 columns, so that a
// block's maximum needs shuffles only.  A mean of squares is taken of the
// differences from the mean, in a second pass over the registers.
#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "stream.cuh"

namespace effort {

// E neighbouring values of type T, 16 bytes at a time
template <typename T, int E>
__device__ __forceinline__ void load_run(const T* p, float (&v)[E]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    const uint4 r = *reinterpret_cast<const uint4*>(p + i);
    const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[i + j] = to_float(t[j]);
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_run(T* p, const float (&v)[E]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    alignas(16) T t[V];
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = from_float<T>(v[i + j]);
    *reinterpret_cast<uint4*>(p + i) = *reinterpret_cast<const uint4*>(t);
  }
}

// Where a thread's elements lie: RUN: E neighbours (E = 8 of 16 bits, 4 of 32),
// else 4 elements 32 apart.  A warp covers 32 E columns of a slot.
template <typename T, bool RUN>
struct Lay {
  static constexpr int E = RUN && sizeof(T) == 2 ? 8 : 4;
  static __device__ __forceinline__ int col(int base, int lane, int e) { return base + (RUN ? lane * E + e : e * 32 + lane); }
  // a run is inside the row or outside of it, whole
  static __device__ __forceinline__ void load(const T* row, int base, int lane, int n, float (&v)[E]) {
    if constexpr (RUN) {
      if (base + lane * E < n) load_run<T, E>(row + base + lane * E, v);
      else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = col(base, lane, e) < n ? to_float(row[col(base, lane, e)]) : 0.0f;
    }
  }
  template <typename U>
  static __device__ __forceinline__ void store(U* row, int base, int lane, int n, const float (&v)[E]) {
    if constexpr (RUN) {
      if (base + lane * E < n) store_run<U, E>(row + base + lane * E, v);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (col(base, lane, e) < n) row[col(base, lane, e)] = from_float<U>(v[e]);
    }
  }
  // weights of a type known at run time
  static __device__ __forceinline__ void load_as(const void* row, int dt, int base, int lane, int n, float (&v)[E]) {
    if constexpr (RUN) {
      if (base + lane * E >= n) return;
      const int c = base + lane * E;
      if (dt == kF32) load_run<float, E>(static_cast<const float*>(row) + c, v);
      else if constexpr (E == 8) {
        if (dt == kF16) load_run<__half, E>(static_cast<const __half*>(row) + c, v);
        else load_run<__nv_bfloat16, E>(static_cast<const __nv_bfloat16*>(row) + c, v);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = load_dt(row, dt, c + e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (col(base, lane, e) < n) v[e] = load_dt(row, dt, col(base, lane, e));
    }
  }
};

// W warps, S slots: a block holds rows of up to 32 E W S columns.
template <typename T, bool RUN, int W, int S>
__global__ void __launch_bounds__(W * 32) k_block_norm(const effort_block_norm_t a) {
  using L = Lay<T, RUN>;
  constexpr int E = L::E;
  __shared__ float red[2][W];
  const int lane = threadIdx.x & 31, warp = warp_index(), n = (int)a.dim;
  const float inv_n = __fdiv_rn(1.0f, (float)n);
  int flip = 0;
  // over the block; the two halves of red in turn: one barrier each
  auto sum = [&](float v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
    if constexpr (W == 1) return v;
    if (lane == 0) red[flip][warp] = v;
    __syncthreads();
    v = lane < W ? red[flip][lane] : 0.0f;
#pragma unroll
    for (int m = W / 2; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
    flip ^= 1;
    return __shfl_sync(~0u, v, 0);
  };
  auto base = [&](int s) { return (s * W + warp) * 32 * E; };
  auto norm = [&](float (&v)[S][E], int kind, const void* w, const void* b) {
    if (kind == EFFORT_NORM_LAYER) {
      float t = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e) t += v[s][e];
      const float mean = sum(t) * inv_n;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (L::col(base(s), lane, e) < n) v[s][e] -= mean;
    }
    float t = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) t += v[s][e] * v[s][e];
    const float r = rsqrtf(sum(t) * inv_n + a.eps);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      float f[E] = {};
      if (w) L::load_as(w, a.weight_dtype, base(s), lane, n, f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[s][e] *= w ? r * (a.weight_offset + f[e]) : r;
      if (b) {
        float o[E] = {};
        L::load_as(b, a.weight_dtype, base(s), lane, n, o);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] += o[e];
      }
    }
  };

  grid_dep_launch();
  grid_dep_wait();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float v[S][E];
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    if (a.y) {
      const T* y = static_cast<const T*>(a.y) + r * a.y_stride;
      float xv[S][E];
#pragma unroll
      for (int s = 0; s < S; ++s) L::load(y, base(s), lane, n, v[s]);
#pragma unroll
      for (int s = 0; s < S; ++s) L::load(x, base(s), lane, n, xv[s]);
      if (a.post_kind != EFFORT_NORM_NONE) norm(v, a.post_kind, a.post_weight, a.post_bias);
      if (a.gate) {
        const T* g = static_cast<const T*>(a.gate) + r * a.gate_stride;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float f[E];
          L::load(g, base(s), lane, n, f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] *= f[e];
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e)
          v[s][e] = L::col(base(s), lane, e) < n ? a.residual_scale * xv[s][e] + a.branch_scale * v[s][e] : 0.0f;
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        L::load(x, base(s), lane, n, v[s]);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] *= a.residual_scale;
      }
    }
    if (a.x_out) {
      T* o = static_cast<T*>(a.x_out) + r * a.x_out_stride;
#pragma unroll
      for (int s = 0; s < S; ++s) L::store(o, base(s), lane, n, v[s]);
    }
    if (a.pre_kind != EFFORT_NORM_NONE) norm(v, a.pre_kind, a.pre_weight, a.pre_bias);
    if (a.h_out) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const long long o = r * a.h_stride;
        if (a.h_dtype == kF32) L::store(static_cast<float*>(a.h_out) + o, base(s), lane, n, v[s]);
        else if constexpr (!RUN || E == 8) {
          if (a.h_dtype == kF16) L::store(static_cast<__half*>(a.h_out) + o, base(s), lane, n, v[s]);
          else L::store(static_cast<__nv_bfloat16*>(a.h_out) + o, base(s), lane, n, v[s]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (L::col(base(s), lane, e) < n) store_dt(a.h_out, a.h_dtype, o + L::col(base(s), lane, e), v[s][e]);
        }
      }
    }
    if (a.q_out) {
      uint8_t* q = static_cast<uint8_t*>(a.q_out) + r * a.q_stride;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (base(s) >= n) break;
        float m = 0.0f;
        bool nan = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (L::col(base(s), lane, e) >= n) v[s][e] = 0.0f;
          m = fmaxf(m, fabsf(v[s][e]));
          nan |= v[s][e] != v[s][e];
        }
        if (nan) m = __int_as_float(0x7fffffff);  // above inf as an integer: it wins the maximum
        int mi = __float_as_int(m);
        constexpr int kLanes = kBlk / E;  // lanes of a block of 128
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) mi = max(mi, __shfl_xor_sync(~0u, mi, d));
        const float scale = __fdiv_rn(__int_as_float(mi), kE4M3Max);
        const int c0 = RUN ? base(s) + lane / kLanes * kBlk : base(s);
        if (lane % kLanes == 0 && c0 < n) a.q_scales[r * a.q_scales_stride + c0 / kBlk] = scale;
        uint32_t b[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
          b[e] = __nv_cvt_float_to_fp8(scale == 0.0f ? 0.0f : __fdiv_rn(v[s][e], scale), __NV_SATFINITE, __NV_E4M3);
        if constexpr (RUN) {
          // q's rows need not start on whole words
          uint8_t* p = q + base(s) + lane * E;
          if (base(s) + lane * E < n) {
            if (((uintptr_t)p & (E - 1)) == 0) {
#pragma unroll
              for (int e = 0; e < E; e += 4)
                *reinterpret_cast<uint32_t*>(p + e) = b[e] | b[e + 1] << 8 | b[e + 2] << 16 | b[e + 3] << 24;
            } else {
#pragma unroll
              for (int e = 0; e < E; ++e) p[e] = (uint8_t)b[e];
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (L::col(base(s), lane, e) < n) q[L::col(base(s), lane, e)] = (uint8_t)b[e];
        }
      }
    }
  }
}

template <typename T, bool RUN, int W, int ES>
static cudaError_t go(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  constexpr int S = ES / Lay<T, RUN>::E;
  // enough blocks for the rows, at most what is resident at once (2048 threads an SM)
  const long long most = (long long)sms * (2048 / (W * 32) < 32 ? 2048 / (W * 32) : 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows < most ? a.rows : most));
  cfg.blockDim = dim3(W * 32);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_block_norm<T, RUN, W, S>, a);
}

// the smallest block that holds a row
template <typename T, bool RUN>
static cudaError_t by_dim(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  if (a.dim <= 256) return go<T, RUN, 1, 8>(a, sms, s);
  if (a.dim <= 1024) return go<T, RUN, 4, 8>(a, sms, s);
  if (a.dim <= 2048) return go<T, RUN, 8, 8>(a, sms, s);
  if (a.dim <= 4096) return go<T, RUN, 8, 16>(a, sms, s);
  if (a.dim <= 8192) return go<T, RUN, 16, 16>(a, sms, s);
  if (a.dim <= 16384) return go<T, RUN, 16, 32>(a, sms, s);
  return go<T, RUN, 32, 40>(a, sms, s);
}

template <typename T>
static cudaError_t by_alignment(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  // runs of 16 bytes: rows of whole runs that start on 16-byte boundaries
  // (runs of 8 values also where h or the weights are fp32)
  constexpr int E = Lay<T, true>::E;
  auto row = [&](const void* p, int64_t stride, size_t size) {
    return !p || (((uintptr_t)p & 15) == 0 && (stride * size) % 16 == 0);
  };
  const size_t wsz = a.weight_dtype == kF32 ? 4 : 2, hsz = a.h_dtype == kF32 ? 4 : 2;
  const bool run = a.dim % E == 0 && row(a.x, a.x_stride, sizeof(T)) && row(a.y, a.y_stride, sizeof(T)) &&
                   row(a.gate, a.gate_stride, sizeof(T)) && row(a.x_out, a.x_out_stride, sizeof(T)) &&
                   row(a.h_out, a.h_stride, hsz) && row(a.post_weight, 0, wsz) && row(a.post_bias, 0, wsz) &&
                   row(a.pre_weight, 0, wsz) && row(a.pre_bias, 0, wsz);
  return run ? by_dim<T, true>(a, sms, s) : by_dim<T, false>(a, sms, s);
}

cudaError_t launch_block_norm(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  if (a.dtype == kF32) return by_alignment<float>(a, sms, s);
  if (a.dtype == kF16) return by_alignment<__half>(a, sms, s);
  return by_alignment<__nv_bfloat16>(a, sms, s);
}

}  // namespace effort
