// The step between two blocks of a decoder layer: norm of the block's output,
// gate, scaled residual, norm for the next block, and its e4m3 quantisation.
//
//   u = post(y);  x' = a x + b g u;  h = pre(x');  s = max|h| over 128 / 448, q = h / s
//
// Bound by its bytes: every input is read once and every output written once,
// and a row stays in its block's registers in between.  One block per row, rows in
// turn: loaded as they are needed where there are few (k_block_norm), two rows ahead
// through shared memory where there are many (k_block_norm_rows).  A warp owns whole
// blocks of 128 columns, so that a block's maximum needs shuffles only.  A mean of squares is taken of the
// differences from the mean, in a second pass over the registers.
#include <atomic>
#include <type_traits>

#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "stream.cuh"

namespace effort {

constexpr int kRowsSmem = 200 * 1024;  // two rows' inputs of a block, at most 2 x 3 x 32 KB

// E neighbouring values of type T, 16 bytes at a time
template <typename T, int E>
__device__ __forceinline__ void load_run(const T* p, float (&v)[E]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    const uint4 r = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (V == 4) v[i + j] = __uint_as_float(w[j]);
      else {
        const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(w[j]);
        v[i + 2 * j] = f.x;
        v[i + 2 * j + 1] = f.y;
      }
    }
  }
}
template <typename T, int E>
__device__ __forceinline__ void store_run(T* p, const float (&v)[E]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < E; i += V) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (V == 4) w[j] = __float_as_uint(v[i + j]);
      else w[j] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[i + 2 * j], v[i + 2 * j + 1]);
    }
    *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Where a thread's elements lie: RUN: E neighbours (E = 8 of 16 bits, 4 of 32),
// else 4 elements 32 apart.  A warp covers 32 E columns of a slot.
template <typename T, bool RUN>
struct Lay {
  static constexpr int E = RUN && sizeof(T) == 2 ? 8 : 4;
  static __device__ __forceinline__ int col(int base, int lane, int e) { return base + (RUN ? lane * E + e : e * 32 + lane); }
  // U: float, or a type of 16 bits; a run is inside the row or outside of it, whole
  template <typename U>
  static __device__ __forceinline__ void load(const U* row, int base, int lane, int n, float (&v)[E]) {
    if constexpr (RUN) {
      const U* p = row + base + lane * E;
      const bool in = base + lane * E < n;
      if constexpr (E * sizeof(U) % 16 == 0) {
        if (in) load_run<U, E>(p, v);
        else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[e] = 0.0f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = in ? to_float(p[e]) : 0.0f;
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
    if (dt == kF32) load(static_cast<const float*>(row), base, lane, n, v);
    else if (dt == kF16) load(static_cast<const __half*>(row), base, lane, n, v);
    else load(static_cast<const __nv_bfloat16*>(row), base, lane, n, v);
  }
};

// One slot's values (zero behind the row's end) of row r in e4m3, with their blocks' scales.
template <typename L, bool RUN, int E>
__device__ __forceinline__ void quantise(const effort_block_norm_t& a, long long r, int base, int lane, int n,
                                         const float (&v)[E]) {
  uint8_t* q = static_cast<uint8_t*>(a.q_out) + r * a.q_stride;
  // as integers: NaN lies above inf and wins the maximum
  int mi = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) mi = max(mi, __float_as_int(v[e]) & 0x7fffffff);
  constexpr int kLanes = kBlk / E;  // lanes of a block of 128
#pragma unroll
  for (int d = kLanes / 2; d; d >>= 1) mi = max(mi, __shfl_xor_sync(~0u, mi, d));
  const float scale = __fdiv_rn(__int_as_float(mi), kE4M3Max);
  const int c0 = RUN ? base + lane / kLanes * kBlk : base;
  if (lane % kLanes == 0 && c0 < n) a.q_scales[r * a.q_scales_stride + c0 / kBlk] = scale;
  // The quotients by one divisor, correctly rounded: with y the rounded
  // reciprocal, t = h y, and the remainder h - t s, which fused
  // multiply-add gives exactly, t + (h - t s) y is h / s rounded (Markstein's
  // theorem, 1990).  Where remainders could underflow, the division itself.
  const float y = __fdiv_rn(1.0f, scale);
  float t[E];
  if (scale > 1e-25f && scale < 1e25f) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float u = v[e] * y;
      t[e] = fmaf(fmaf(-u, scale, v[e]), y, u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) t[e] = scale == 0.0f ? 0.0f : __fdiv_rn(v[e], scale);
  }
  uint32_t b[E];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(t[e], t[e + 1]), __NV_SATFINITE, __NV_E4M3);
    b[e] = two & 0xff;
    b[e + 1] = two >> 8;
  }
  if constexpr (RUN) {
    // q's rows need not start on whole words
    uint8_t* p = q + base + lane * E;
    if (base + lane * E < n) {
      if (((uintptr_t)p & (E - 1)) == 0) {
        uint32_t w[E / 4];
#pragma unroll
        for (int e = 0; e < E; e += 4) w[e / 4] = b[e] | b[e + 1] << 8 | b[e + 2] << 16 | b[e + 3] << 24;
        if constexpr (E == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) p[e] = (uint8_t)b[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (L::col(base, lane, e) < n) q[L::col(base, lane, e)] = (uint8_t)b[e];
  }
}

// Sums over a block of W warps; the two halves of `red` in turn: one barrier each.
template <int W>
struct BlockSum {
  float (*red)[W];
  int lane, warp, flip;
  __device__ __forceinline__ float operator()(float v) {
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
  }
};

// h to its array, whose type is known at run time
template <typename L, bool RUN, int E>
__device__ __forceinline__ void store_h(const effort_block_norm_t& a, long long r, int base, int lane, int n,
                                        const float (&v)[E]) {
  const long long o = r * a.h_stride;
  if (a.h_dtype == kF32) L::store(static_cast<float*>(a.h_out) + o, base, lane, n, v);
  else if constexpr (!RUN || E == 8) {
    if (a.h_dtype == kF16) L::store(static_cast<__half*>(a.h_out) + o, base, lane, n, v);
    else L::store(static_cast<__nv_bfloat16*>(a.h_out) + o, base, lane, n, v);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (L::col(base, lane, e) < n) store_dt(a.h_out, a.h_dtype, o + L::col(base, lane, e), v[e]);
  }
}

// W warps, S slots: a block holds rows of up to 32 E W S columns.
template <typename T, bool RUN, int W, int S>
__global__ void __launch_bounds__(W * 32) k_block_norm(const effort_block_norm_t a) {
  using L = Lay<T, RUN>;
  constexpr int E = L::E;
  __shared__ float red[2][W];
  const int lane = threadIdx.x & 31, warp = warp_index(), n = (int)a.dim;
  const float inv_n = __fdiv_rn(1.0f, (float)n);
  BlockSum<W> sum{red, lane, warp, 0};
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
    // the type is chosen once for all slots, so that their loads go out together
    auto affine = [&](auto type) {
      using U = decltype(type);
      if (w) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float f[E];
          L::load(static_cast<const U*>(w), base(s), lane, n, f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] *= r * (a.weight_offset + f[e]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] *= r;
      }
      if (b) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float f[E];
          L::load(static_cast<const U*>(b), base(s), lane, n, f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] += f[e];
        }
      }
    };
    if (a.weight_dtype == kF32) affine(0.0f);
    else if (a.weight_dtype == kF16) affine(__half());
    else affine(__nv_bfloat16());
  };

  grid_dep_launch();
  grid_dep_wait();
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    float v[S][E];
    const T* x = static_cast<const T*>(a.x) + r * a.x_stride;
    if (a.y) {
      const T* y = static_cast<const T*>(a.y) + r * a.y_stride;
#pragma unroll
      for (int s = 0; s < S; ++s) L::load(y, base(s), lane, n, v[s]);
      if (a.post_kind != EFFORT_NORM_NONE) norm(v, a.post_kind, a.post_weight, a.post_bias);
      if (a.gate) {
        const T* gate = static_cast<const T*>(a.gate) + r * a.gate_stride;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float g[E];
          L::load(gate, base(s), lane, n, g);
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] *= g[e];
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float f[E];
        L::load(x, base(s), lane, n, f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] = a.residual_scale * f[e] + a.branch_scale * v[s][e];
      }
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
      for (int s = 0; s < S; ++s) store_h<L, RUN, E>(a, r, base(s), lane, n, v[s]);
    }
    if (a.q_out) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (base(s) < n) quantise<L, RUN, E>(a, r, base(s), lane, n, v[s]);
    }
  }
}

// The same for many rows of whole runs: a block takes row after row, its inputs
// two rows ahead in shared memory (bulk copies), and keeps the weights of its
// columns in registers.  With direct loads a row's chain of load, sum, load,
// sum left the memory idle (68 against 53 us at 8192 x 4096 bf16, 106 against 71
// with gate and e4m3).
// KEEP: the weights are of type T.
template <typename T, int W, int S, bool KEEP>
__global__ void __launch_bounds__(W * 32, 24 / W) k_block_norm_rows(const effort_block_norm_t a, const WaitHook hook) {
  using L = Lay<T, true>;
  constexpr int E = L::E;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][W];
  __shared__ uint64_t bars[2];
  __shared__ long long late;  // the row at which the copying thread's wait ran out
  const int lane = threadIdx.x & 31, warp = warp_index(), n = (int)a.dim;
  const float inv_n = __fdiv_rn(1.0f, (float)n);
  const bool gates = a.gate && a.gate_stride != 0;
  const uint32_t bytes = (uint32_t)n * sizeof(T), arrays = 1 + (a.y != nullptr) + gates;
  const uint32_t sbase = smem_u32(smem), bar = smem_u32(bars);
  BlockSum<W> sum{red, lane, warp, 0};
  auto col = [&](int s) { return (s * W + warp) * 32 * E + lane * E; };
  if (threadIdx.x == 0) {
    late = -1;
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  grid_dep_launch();
  grid_dep_wait();
  bool fine = true;  // no wait of this thread has run out
  int asked = 0;
  auto ask = [&](long long r, int st) {  // x, y and the gate's row, one after another
    if (threadIdx.x != 0 || r >= a.rows || !fine) return;
    const uint32_t to = sbase + st * arrays * bytes;
    mbar_expect(bar + 8 * st, arrays * bytes + hook.lost(asked++));
    bulk_load(to, static_cast<const T*>(a.x) + r * a.x_stride, bytes, bar + 8 * st);
    if (a.y) bulk_load(to + bytes, static_cast<const T*>(a.y) + r * a.y_stride, bytes, bar + 8 * st);
    if (gates) bulk_load(to + (arrays - 1) * bytes, static_cast<const T*>(a.gate) + r * a.gate_stride, bytes, bar + 8 * st);
  };
  ask(blockIdx.x, 0);
  ask(blockIdx.x + (long long)gridDim.x, 1);
  // weights of this thread's columns stay in registers as they are; those of
  // another type than the rows' are read again for every row
  constexpr int H = KEEP ? E * (int)sizeof(T) / 4 : 1;
  uint32_t wp[S][H], wn[S][H];
  auto hold = [&](const void* w, uint32_t (&h)[S][H]) {
    if constexpr (KEEP) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < H; ++i)
          h[s][i] = w && col(s) < n ? static_cast<const uint32_t*>(w)[col(s) * (int)sizeof(T) / 4 + i] : 0u;
    }
  };
  hold(a.post_weight, wp);
  hold(a.pre_weight, wn);
  auto norm = [&](float (&v)[S][E], int kind, const void* w, const uint32_t (&h)[S][H], const void* b) {
    if (kind == EFFORT_NORM_LAYER) {
      float t = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e) t += v[s][e];
      const float mean = sum(t) * inv_n;
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (col(s) < n) {
#pragma unroll
          for (int e = 0; e < E; ++e) v[s][e] -= mean;
        }
    }
    float t = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) t += v[s][e] * v[s][e];
    const float r = rsqrtf(sum(t) * inv_n + a.eps), ro = r * a.weight_offset;
    if (!w) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] *= r;
    } else if constexpr (KEEP) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          if constexpr (sizeof(T) == 4) v[s][i] *= fmaf(r, __uint_as_float(h[s][i]), ro);
          else {
            const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(h[s][i]);
            v[s][2 * i] *= fmaf(r, f.x, ro);
            v[s][2 * i + 1] *= fmaf(r, f.y, ro);
          }
        }
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float f[E] = {};
        L::load_as(w, a.weight_dtype, col(s) - lane * E, lane, n, f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] *= fmaf(r, f[e], ro);
      }
    }
    if (b) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float o[E] = {};
        L::load_as(b, a.weight_dtype, col(s) - lane * E, lane, n, o);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] += o[e];
      }
    }
  };
  int st = 0, ph = 0;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    fine = fine && mbar_wait(bar + 8 * st, ph, hook.tries);
    const T* in = reinterpret_cast<const T*>(smem + st * arrays * bytes);
    float v[S][E];
    // one array's values of slot s
    auto get = [&](int array, int s, float (&f)[E]) {
      if (col(s) < n) load_run<T, E>(in + (size_t)array * n + col(s), f);
      else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = 0.0f;
      }
    };
    if (a.y) {
#pragma unroll
      for (int s = 0; s < S; ++s) get(1, s, v[s]);
      if (a.post_kind != EFFORT_NORM_NONE) norm(v, a.post_kind, a.post_weight, wp, a.post_bias);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float f[E], g[E];
        get(0, s, f);
        if (gates) get(2, s, g);
        else if (a.gate) L::load(static_cast<const T*>(a.gate), col(s) - lane * E, lane, n, g);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (a.gate) v[s][e] *= g[e];
          v[s][e] = a.residual_scale * f[e] + a.branch_scale * v[s][e];
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        get(0, s, v[s]);
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] *= a.residual_scale;
      }
    }
    if (!fine) {
      if (threadIdx.x == 0 && late < 0) late = r;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int e = 0; e < E; ++e) v[s][e] = __int_as_float(0x7fffffff);
    }
    if (a.x_out) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (col(s) < n) store_run<T, E>(static_cast<T*>(a.x_out) + r * a.x_out_stride + col(s), v[s]);
    }
    // every thread has read the row: its place is free for the row after the next
    if (a.pre_kind != EFFORT_NORM_NONE) norm(v, a.pre_kind, a.pre_weight, wn, a.pre_bias);
    else __syncthreads();
    ask(r + 2ll * gridDim.x, st);
    if (a.h_out) {
#pragma unroll
      for (int s = 0; s < S; ++s) store_h<L, true, E>(a, r, col(s) - lane * E, lane, n, v[s]);
    }
    if (a.q_out) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (col(s) - lane * E < n) quantise<L, true, E>(a, r, col(s) - lane * E, lane, n, v[s]);
    }
    ph ^= st;
    st ^= 1;
  }
  // copies in flight end before the block does
  if (threadIdx.x == 0 && !fine) {
    const int k = (int)((late - blockIdx.x) / gridDim.x);  // that row among the block's: it and the next were asked for
    for (int i = k; i < k + 2 && blockIdx.x + (long long)gridDim.x * i < a.rows; ++i)
      mbar_wait(bar + 8 * (i & 1), i >> 1 & 1, hook.tries);
  }
}

template <typename T, int W, int ES, bool KEEP>
static cudaError_t go_rows_as(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  constexpr int S = ES / Lay<T, true>::E;
  const size_t smem = 2 * (size_t)a.dim * sizeof(T) * (1 + (a.y != nullptr) + (a.gate && a.gate_stride != 0));
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!done[dev].load()) {
    e = cudaFuncSetAttribute(k_block_norm_rows<T, W, S, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    if (e != cudaSuccess) return e;
    done[dev].store(true);
  }
  // blocks resident at once, by threads and by shared memory
  const int by_smem = (int)(kSmemMax / (smem + 2048));
  const long long most = (long long)sms * (24 / W < by_smem ? 24 / W : by_smem < 1 ? 1 : by_smem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows < most ? a.rows : most));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_block_norm_rows<T, W, S, KEEP>, a, wait_hook());
}

template <typename T, int W, int ES>
static cudaError_t go_rows(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  constexpr int kT = sizeof(T) == 4 ? kF32 : std::is_same_v<T, __half> ? kF16 : kBF16;
  return a.weight_dtype == kT ? go_rows_as<T, W, ES, true>(a, sms, s) : go_rows_as<T, W, ES, false>(a, sms, s);
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
  return go<T, RUN, 16, 80>(a, sms, s);
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
  if (!run) return by_dim<T, false>(a, sms, s);
  // rows in turn pay from a few for each block on (one row: 3.7 us direct); of
  // rows that leave an SM one block only, from the second on (34 against 18 us
  // at 308 x 13888 bf16 with gate and e4m3)
  if (a.rows >= (a.dim > 8192 ? 1 : 4) * (long long)sms && a.dim > 256) {
    if (a.dim <= 1024) return go_rows<T, 2, 16>(a, sms, s);
    if (a.dim <= 2048) return go_rows<T, 4, 16>(a, sms, s);
    if (a.dim <= 4096) return go_rows<T, 8, 16>(a, sms, s);
    if (a.dim <= 8192) return go_rows<T, 16, 16>(a, sms, s);
    if (a.dim <= 16384 && sizeof(T) == 2) return go_rows<T, 16, 32>(a, sms, s);
  }
  return by_dim<T, true>(a, sms, s);
}

cudaError_t launch_block_norm(const effort_block_norm_t& a, int sms, cudaStream_t s) {
  if (a.dtype == kF32) return by_alignment<float>(a, sms, s);
  if (a.dtype == kF16) return by_alignment<__half>(a, sms, s);
  return by_alignment<__nv_bfloat16>(a, sms, s);
}

}  // namespace effort
