// The product with e4m3 operands and one scale for each block of 128:
//
//   out[r][n] = sum_b xs[r][b] ws[b][n / 128] sum_{k in b} x[r][k] w[k][n]
//
// and the layout of its weights.
#include <atomic>

#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "stream.cuh"

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

// ---------------------------------------------------------------- few rows
// rows <= 8 NT of x against all of w: the weights' stream of stream.cuh.  The
// 16-row tiles are dealt to clusters in even, contiguous shares; the blocks of
// a cluster share the tiles' K blocks and join their sums through distributed
// shared memory, so there is no scratch and no order that varies.
struct FewRows {
  TileMat w;
  const float* ws;
  int nsb, I, O, rows;
  const uint8_t* x;
  long long xstride;
  const float* xs;
  long long xsstride;
  void* out;
  long long ostride;
  int odt, tiles, cluster, kw;
};

template <int NT>
struct FewRowsCfg {
  static constexpr int kMT = NT == 4 ? 2 : 4;      // tiles of a group
  static constexpr int kStages = NT == 4 ? 5 : 3;  // 20 or 24 KB of ring for each warp
  static constexpr int kStageBytes = kMT * 2 * kCoreBytes;
  static constexpr int kPitch = kMT * 16 + 4;      // floats of one column in the join; + 4: no bank met twice
  static constexpr int kRed = NT * 8 * kPitch;     // floats of one warp's part
  static constexpr size_t kBars = 0, kRing = 1024, kRedAt = kRing + (size_t)kSWarps * kStages * kStageBytes;
  static constexpr size_t kSmem = kRedAt + (size_t)kSWarps * kRed * 4;
  static_assert(kSmem <= 227 * 1024, "one block per SM");
};

template <int NT>
__global__ void __launch_bounds__(kSThreads, 1) k_fp8_few_rows(const FewRows a) {
  using C = FewRowsCfg<NT>;
  constexpr int MT = C::kMT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float* red = reinterpret_cast<float*>(smem + C::kRedAt);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int cl = a.cluster, rank = cl > 1 ? (int)cluster_rank() : 0;
  const int ncl = gridDim.x / cl, c = blockIdx.x / cl;
  const int t0 = (int)((long long)a.tiles * c / ncl), t1 = (int)((long long)a.tiles * (c + 1) / ncl);
  const int kb0 = a.w.nkb * rank / cl, kb1 = a.w.nkb * (rank + 1) / cl;
  const int kw = a.kw, rw = kSWarps / kw, wk = warp % kw, wr = warp / kw;
  const int groups = cdiv(t1 - t0, MT);
  const size_t core_stride = (size_t)a.w.nkb * kCoreBytes;

  Ring<C::kStages, C::kStageBytes> ring;
  ring.init(sbase + C::kRing, sbase + C::kBars, warp, lane);
  // the warp's list: groups wr, wr + rw, ..; in each the K blocks kb0 + wk, + kw, ..
  int pg = wr, pk = kb0 + wk;
  auto ask = [&]() {
    if (pk >= kb1) return;  // no K block for this warp
    if (pg >= groups) return;
    const int t = t0 + pg * MT, n = min(MT, t1 - t);
    ring.fill(a.w.data + ((size_t)(2 * t) * a.w.nkb + pk) * kCoreBytes, 2 * n, core_stride, lane);
    pk += kw;
    if (pk >= kb1) {
      pk = kb0 + wk;
      pg += rw;
    }
  };
  // the weights do not depend on the kernel before
#pragma unroll
  for (int s = 0; s < C::kStages; ++s) ask();
  grid_dep_launch();
  grid_dep_wait();

  const int live = NT == 1 ? 1 : (a.rows + 7) / 8;
  bool fine = true;
  for (int gi = wr; gi < groups; gi += rw) {
    const int t = t0 + gi * MT, n = min(MT, t1 - t);
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    for (int kb = kb0 + wk; kb < kb1; kb += kw) {
      // B: column g of each tile is a row of x, elements 32 q .. 32 q + 31
      uint32_t b[1][NT][8][2];
      float sx[NT][2], sw[MT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint4 v[2] = {};
        const int r = 8 * j + g;
        if (r < a.rows) {
          const uint8_t* p = a.x + r * a.xstride;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = kb * kBlk + 32 * q + 16 * h;
            if (k < a.I) v[h] = __ldg(reinterpret_cast<const uint4*>(p + k));
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = 8 * j + 2 * q + e;
          sx[j][e] = rr < a.rows ? __ldg(a.xs + rr * a.xsstride + kb) : 0.0f;
        }
        if (kb == a.w.nkb - 1) {  // bytes behind the row's end count as zero
          uint8_t* y = reinterpret_cast<uint8_t*>(v);
          const int k = kb * kBlk + 32 * q;
#pragma unroll
          for (int h = 0; h < 32; ++h)
            if (k + h >= a.I) y[h] = 0;
        }
        const uint32_t u[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          b[0][j][s][0] = e4m3x2_to_half2(u[s]);
          b[0][j][s][1] = e4m3x2_to_half2(u[s] >> 16);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) sw[m] = __ldg(a.ws + (size_t)kb * a.nsb + min((t + m) / 8, a.nsb - 1));
      uint32_t at;
      fine &= ring.wait(&at);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m < n) {
          float d[NT][4] = {};
          mma_tile<kWE4M3, NT, 1, 8>(at + m * 2 * kCoreBytes, g, q, b, live, d);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(d[j][e] * sx[j][e & 1], sw[m], acc[m][j][e]);
        }
      }
      __syncwarp();  // every lane has read the stage
      ask();
    }
    // join the warps' sums (and the cluster's)
    named_sync(1 + wr, kw * 32);
    float* mine = red + warp * C::kRed;
    const float poison = fine ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * q + (e & 1)) * C::kPitch + 16 * m + g + 8 * (e >> 1)] = acc[m][j][e] + poison;
    named_sync(1 + wr, kw * 32);
    const int outs = n * 16 * a.rows;
    float* first = red + wr * kw * C::kRed;
    if (cl == 1) {
      for (int i = threadIdx.x - wr * kw * 32; i < outs; i += kw * 32) {
        const int r = i / (n * 16), o = i % (n * 16), col = t * 16 + o;
        float s = 0.0f;
        for (int w = 0; w < kw; ++w) s += first[w * C::kRed + r * C::kPitch + o];
        if (col < a.O) store_dt(a.out, a.odt, r * a.ostride + col, s);
      }
    } else {
      // kw = 8, rw = 1: the block's sum into the first warp's part, then each
      // block takes its share of the outputs
      for (int i = threadIdx.x; i < outs; i += kSThreads) {
        const int at = i / (n * 16) * C::kPitch + i % (n * 16);
        float s = 0.0f;
        for (int w = 0; w < kSWarps; ++w) s += red[w * C::kRed + at];
        red[at] = s;
      }
      cluster_sync();
      const int i0 = outs * rank / cl, i1 = outs * (rank + 1) / cl;
      for (int i = i0 + threadIdx.x; i < i1; i += kSThreads) {
        const int r = i / (n * 16), o = i % (n * 16), col = t * 16 + o;
        const uint32_t at = sbase + (uint32_t)C::kRedAt + (uint32_t)(r * C::kPitch + o) * 4;
        float s = 0.0f;
        for (int w = 0; w < cl; ++w) s += remote_float(at, w);
        if (col < a.O) store_dt(a.out, a.odt, r * a.ostride + col, s);
      }
      cluster_sync();  // the sums may be written over (and, at the end, the block may leave)
    }
  }
}

// Blocks of `cluster` that fit the device at once (one block per SM).
template <int NT>
static int few_rows_clusters(int cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = FewRowsCfg<NT>::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k_fp8_few_rows<NT>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

template <int NT>
static cudaError_t launch_few_rows(FewRows a, cudaStream_t s) {
  // per device, looked up once: the blocks that fit for each cluster size
  static std::atomic<int> fit[kMaxDevices][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (fit[dev][0].load() == 0) {
    e = cudaFuncSetAttribute(k_fp8_few_rows<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FewRowsCfg<NT>::kSmem);
    if (e != cudaSuccess) return e;
    for (int i = 3; i >= 0; --i) fit[dev][i].store(few_rows_clusters<NT>(1 << i));
    if (fit[dev][0].load() < 1) return cudaErrorLaunchOutOfResources;
  }
  // the cluster size whose longest share (tiles x K blocks of one block) is
  // shortest; a wider one has to win by 2% to pay for its joins
  long long best = 0;
  int ncl = 0;
  for (int i = 0; i < 4; ++i) {
    const int cl = 1 << i, n = min(fit[dev][i].load(), a.tiles);
    if (n < 1 || cl > a.w.nkb) break;
    const long long cost = (long long)cdiv(a.tiles, n) * cdiv(a.w.nkb, cl);
    if (ncl == 0 || cost * 102 < best * 100) {
      best = cost;
      a.cluster = cl;
      ncl = n;
    }
  }
  a.kw = kSWarps;
  if (a.cluster == 1)
    while (a.kw > a.w.nkb) a.kw /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ncl * a.cluster));
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = FewRowsCfg<NT>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)a.cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp8_few_rows<NT>, a);
}

cudaError_t launch_fp8_matmul(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                              const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                              cudaStream_t s) {
  const size_t osz = odt == kF32 ? 4 : 2;
  for (int64_t r = 0; r < rows; r += 32) {
    FewRows a = {w, ws, cdiv(O, kBlk), I, O, (int)(rows - r < 32 ? rows - r : 32), x + r * xstride, xstride,
                 xs + r * xsstride, xsstride, (char*)out + r * ostride * osz, ostride, odt, cdiv(O, 16), 1, kSWarps};
    cudaError_t e = a.rows <= 8 ? launch_few_rows<1>(a, s) : a.rows <= 16 ? launch_few_rows<2>(a, s) : launch_few_rows<4>(a, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace effort
