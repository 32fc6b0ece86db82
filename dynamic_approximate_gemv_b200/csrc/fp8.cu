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
    *reinterpret_cast<uint4*>(out + mat * stride + core_at(core, kb, nkb) + r * 128 + ((ch ^ r) << 4)) =
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
  const float* ws;   // [row block][K block], rows of nkb4 floats
  int nkb4, I, O, rows;
  const uint8_t* x;
  long long xstride;
  const float* xs;
  long long xsstride;
  void* out;
  long long ostride;
  int odt, tiles, cluster, kw;
  WaitHook hook;
};
constexpr int kFewRowsMax = 16;
constexpr int kFewExtra = 12 * 1024;  // the table of x's scales
template <int NT>
using FewShape = StreamShape<NT * 8, 128, 16, kFewExtra>;

template <int NT>
__global__ void __launch_bounds__(FewShape<NT>::kThreads, 1) k_fp8_few_rows(const FewRows a) {
  using S = FewShape<NT>;
  constexpr int MT = S::kMT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float* red = reinterpret_cast<float*>(smem + S::kRedAt);
  const uint32_t xtab = sbase + S::kExtraAt;  // x_scales of the block's K blocks: [K block][NT * 8]
  const int lane = threadIdx.x & 31, warp = warp_index(), g = lane >> 2, q = lane & 3;
  const int cl = a.cluster, rank = cluster_rank();
  const int ncl = gridDim.x / cl, c = blockIdx.x / cl;
  const int t0 = (int)((long long)a.tiles * c / ncl), t1 = (int)((long long)a.tiles * (c + 1) / ncl);
  const int kb0 = a.w.nkb * rank / cl, kb1 = a.w.nkb * (rank + 1) / cl;
  const int kw = a.kw, rw = S::kWarps / kw, wk = warp % kw, wr = warp / kw;
  // (cut at multiples of MT, so that a group never spans 64 stored rows, some
  // shares would have a group more: 14.4 against 11.7 us at 14336 x 4096)
  const int groups = cdiv(t1 - t0, MT);

  Ring<S> ring;
  ring.init(sbase, warp, lane);
  // A stage: the cores and the scales (they do not depend on the kernel
  // before), then the rows of x.  The warp's list: groups wr, wr + rw, ..; in
  // each the K blocks kb0 + wk, + kw, ..
  auto ask_weights = [&](int gi, int kb) {
    const int t = t0 + gi * MT, n = min(MT, t1 - t);
    const int last = a.I - kb * kBlk, xb = last >= kBlk ? kBlk : (last + 15) / 16 * 16;
    const uint32_t buf = ring.next_buf(), bar = ring.next_bar();
    const int n1 = min(n, 4 - (t & 3));               // tiles up to the end of 64 stored rows
    const bool two = (t + n - 1) / 8 > t / 8;         // whether the tiles lie in two blocks of 128 columns
    if (lane == 0) {
      mbar_expect(bar, n * 2 * kCoreBytes + a.rows * xb + (two ? 32 : 16) + a.hook.lost(ring.put));
      bulk_load(buf, a.w.data + core_at(2 * t, kb, a.w.nkb), n1 * 2 * kCoreBytes, bar);
      if (n1 < n)
        bulk_load(buf + n1 * 2 * kCoreBytes, a.w.data + core_at(2 * (t + n1), kb, a.w.nkb), (n - n1) * 2 * kCoreBytes, bar);
      bulk_load(buf + S::kScaleAt, a.ws + (size_t)(t / 8) * a.nkb4 + (kb & ~3), 16, bar);
      if (two) bulk_load(buf + S::kScaleAt + 16, a.ws + (size_t)(t / 8 + 1) * a.nkb4 + (kb & ~3), 16, bar);
    }
    __syncwarp();
  };
  auto ask_rows = [&](int kb) {
    const int last = a.I - kb * kBlk, xb = last >= kBlk ? kBlk : (last + 15) / 16 * 16;
    const uint32_t buf = ring.next_buf(), bar = ring.next_bar();
    if (lane < a.rows) bulk_load(buf + S::kActAt + lane * S::kRowPitch, a.x + lane * a.xstride + kb * kBlk, xb, bar);
    ++ring.put;
  };
  int pg = wr, pk = kb0 + wk;
  const bool busy = pk < kb1;
  auto step = [&]() {
    pk += kw;
    if (pk >= kb1) {
      pk = kb0 + wk;
      pg += rw;
    }
  };
  // the first stages' weights ahead of the kernel before
  int early = 0;
  for (; early < S::kStages && busy && pg < groups; ++early) {
    ask_weights(pg, pk);
    ++ring.put;
    step();
  }
  grid_dep_launch();
  grid_dep_wait();
  // (plain loads: the kernel before may still have been writing when this one started)
  for (int i = threadIdx.x; i < (kb1 - kb0) * NT * 8; i += S::kThreads) {
    const int r = i / (kb1 - kb0), k = i % (kb1 - kb0);
    const float s = r < a.rows ? a.xs[r * a.xsstride + kb0 + k] : 0.0f;
    *reinterpret_cast<float*>(smem + S::kExtraAt + (k * NT * 8 + r) * 4) = s;
  }
  ring.put = 0;
  for (int i = 0, k = kb0 + wk; i < early; ++i) {
    ask_rows(k);
    k = k + kw < kb1 ? k + kw : kb0 + wk;
  }
  __syncthreads();

  const int live = NT == 1 ? 1 : (a.rows + 7) / 8;
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
      const uint32_t at = ring.wait(smem, warp, a.hook, [&]() { pg = groups; });
      uint32_t b[1][NT][8][2];
      float sx[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        act_e4m3(at + S::kActAt + (8 * j + g) * S::kRowPitch, q, 8 * j + g < a.rows, a.I - kb * kBlk, b[0][j]);
#pragma unroll
        for (int e = 0; e < 2; ++e) sx[j][e] = lds_float(xtab + ((kb - kb0) * NT * 8 + 8 * j + 2 * q + e) * 4);
      }
      const float sw[2] = {lds_float(at + S::kScaleAt + 4 * (kb & 3)), lds_float(at + S::kScaleAt + 16 + 4 * (kb & 3))};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m < n) {
          float d[NT][4] = {};
          mma_tile<kWE4M3, NT, 1, 8>(at + m * 2 * kCoreBytes, g, q, b, live, d);
          const float s = (t + m) / 8 == t / 8 ? sw[0] : sw[1];
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(d[j][e] * sx[j][e & 1], s, acc[m][j][e]);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (busy && pg < groups) {
        ask_weights(pg, pk);
        ask_rows(pk);
        step();
      }
    }
    // join the warps' sums (and the cluster's)
    set_sync(wr, kw);
    float* mine = red + warp * S::kRed;
    const float poison = ring.fine ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * q + (e & 1)) * S::kPitch + 16 * m + g + 8 * (e >> 1)] = acc[m][j][e] + poison;
    set_sync(wr, kw);
    const int outs = n * 16 * a.rows;
    float* first = red + wr * kw * S::kRed;
    if (cl == 1) {
      for (int i = threadIdx.x - wr * kw * 32; i < outs; i += kw * 32) {
        const int r = i / (n * 16), o = i % (n * 16), col = t * 16 + o;
        float s = 0.0f;
        for (int w = 0; w < kw; ++w) s += first[w * S::kRed + r * S::kPitch + o];
        if (col < a.O) store_dt(a.out, a.odt, r * a.ostride + col, s);
      }
    } else {
      // one set of warps: the block's sum into the first warp's part, then each
      // block takes its share of the outputs
      for (int i = threadIdx.x; i < outs; i += S::kThreads) {
        const int at = i / (n * 16) * S::kPitch + i % (n * 16);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < S::kWarps; ++w) s += red[w * S::kRed + at];
        red[at] = s;
      }
      cluster_sync();
      const int i0 = outs * rank / cl, i1 = outs * (rank + 1) / cl;
      for (int i = i0 + threadIdx.x; i < i1; i += S::kThreads) {
        const int r = i / (n * 16), o = i % (n * 16), col = t * 16 + o;
        const uint32_t at = sbase + (uint32_t)S::kRedAt + (uint32_t)(r * S::kPitch + o) * 4;
        float s = 0.0f;
        for (int w = 0; w < cl; ++w) s += remote_float(at, w);
        if (col < a.O) store_dt(a.out, a.odt, r * a.ostride + col, s);
      }
      cluster_sync();  // the sums may be written over (and, at the end, the block may leave)
    }
  }
  ring.drain(smem, warp, lane, a.hook);
}

// Blocks of `cluster` that fit the device at once (one block per SM).
template <int NT>
static int few_rows_clusters(int cluster) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3(FewShape<NT>::kThreads);
  cfg.dynamicSmemBytes = FewShape<NT>::kSmem;
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
    e = cudaFuncSetAttribute(k_fp8_few_rows<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FewShape<NT>::kSmem);
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
    if ((long long)cdiv(a.w.nkb, cl) * NT * 8 * 4 > kFewExtra) continue;  // the table of x's scales
    const long long per = cdiv(a.tiles, n);
    const long long cost = per * cdiv(a.w.nkb, cl) + (cl > 1 ? 24 * cdiv(per, FewShape<NT>::kMT) : 0);
    if (ncl == 0 || cost * 102 < best * 100) {
      best = cost;
      a.cluster = cl;
      ncl = n;
    }
  }
  if (ncl == 0) return cudaErrorInvalidConfiguration;
  a.kw = FewShape<NT>::kWarps;
  if (a.cluster == 1)
    while (a.kw > a.w.nkb) a.kw /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ncl * a.cluster));
  cfg.blockDim = dim3(FewShape<NT>::kThreads);
  cfg.dynamicSmemBytes = FewShape<NT>::kSmem;
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

cudaError_t launch_fp8_tc(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                          const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                          cudaStream_t s);

cudaError_t launch_fp8_matmul(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                              const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                              cudaStream_t s) {
  // Few rows stream through registers, with the least to set up: up to 8, and
  // up to 16 of small matrices.  A wide and large matrix fills the tensor cores'
  // tiles at once.  Measured, stream / tensor cores in us, in x out:
  //   rows           2           8           9           16
  //   512 x 512      1.9 / 2.9   2.1 / 3.0   2.6 / 3.0   2.8 / 3.2
  //   1024 x 2048    2.8 / 3.9   3.0 / 4.0   3.0 / 4.1   3.3 / 4.2
  //   4096 x 1024    3.1 / 5.8   3.6 / 6.3   5.8 / 6.3   6.7 / 6.4
  //   2048 x 4096    3.7 / 6.5   4.0 / 6.7   4.9 / 6.7   5.4 / 6.7
  //   4096 x 4096    5.2 / 8.3   5.7 / 8.5   7.7 / 8.5   8.7 / 8.6
  //   4096 x 8192    8.4 / 10.5  9.3 / 10.7  10.1 / 10.6 11.3 / 10.7
  //   2048 x 16384   9.2 / 9.0   10.3 / 9.4  10.9 / 9.5  12.5 / 9.6
  //   4096 x 14336   13.2 / 13.0 15.1 / 13.2 17.0 / 13.2 19.6 / 13.5
  //   14336 x 4096   11.4 / 14.5 13.2 / 14.7 21.7 / 14.7 24.8 / 14.7
  //   8192 x 28672   41.6 / 43.0 44.3 / 43.1 55.5 / 43.1 64.4 / 43.7
  // So the rule gives up to 2 us away where 9 to 12 rows meet 4 to 32 M weights, and
  // where 2 to 8 rows meet 32 M that are just twice as wide as long.
  const long long size = (long long)I * O;
  const bool wide = rows > 1 && O >= 2 * I && size >= 32ll << 20;
  if (wide || rows > kFewRowsMax || (rows > 8 && size > 2ll << 20))
    return launch_fp8_tc(w, ws, I, O, x, xstride, xs, xsstride, rows, odt, out, ostride, s);
  const size_t osz = odt == kF32 ? 4 : 2;
  // 16 rows' scales of a very long K do not fit beside the ring: 8 rows then
  const int most = w.nkb > 1536 ? 8 : kFewRowsMax;
  for (int64_t r = 0; r < rows; r += most) {
    FewRows a = {w, ws, align4(w.nkb), I, O, (int)(rows - r < most ? rows - r : most), x + r * xstride,
                 xstride, xs + r * xsstride, xsstride, (char*)out + r * ostride * osz, ostride, odt, cdiv(O, 16), 1, 1, wait_hook()};
    cudaError_t e = a.rows <= 8 ? launch_few_rows<1>(a, s) : launch_few_rows<2>(a, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// Scales [in block][out block] as the products take them: [matrix][out block][in
// block], rows of align4(in blocks) floats, so that 16 bytes hold four K blocks.
__global__ void k_turn_scales(const float* s, int nkb, int nsb, float* out) {
  const size_t m = blockIdx.y;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < nsb * align4(nkb); i += gridDim.x * blockDim.x) {
    const int b = i / align4(nkb), k = i % align4(nkb);
    out[m * nsb * align4(nkb) + i] = k < nkb ? s[(m * nkb + k) * nsb + b] : 0.0f;
  }
}
cudaError_t launch_turn_scales(const float* s, int mats, int nkb, int nsb, float* out, cudaStream_t st) {
  k_turn_scales<<<dim3(64, (unsigned)mats), 256, 0, st>>>(s, nkb, nsb, out);
  return cudaGetLastError();
}

}  // namespace effort
