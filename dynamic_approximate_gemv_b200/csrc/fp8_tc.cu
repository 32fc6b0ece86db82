// The product with e4m3 operands on the tensor cores (tcgen05):
//
//   out[r][n] = sum_b xs[r][b] ws[b][n / 128] sum_{k in b} x[r][k] w[k][n]
//
// Each K block of 128 is one accumulation of four matrix instructions in tensor
// memory; the epilogue warps read it, multiply by the block's scales and add
// it in fp32 registers while the next blocks are multiplied.
//
// Which operand takes the instruction's M side (the lanes of tensor memory):
// for few rows the weights, so that x needs only N = 16, 32 or 64 columns;
// else the rows of x, so that an epilogue thread holds one row and needs one
// scale for each K block (with the weights there it needs one for each column:
// 2300 clocks a K block of 128 x 256 against the instruction's 512).
//
// Roles: warp 0 copies (the weights' cores as they are stored, x through a
// tensor map), warp 1 issues the matrix instructions, warp 2 turns the scales
// of eight K blocks at a time into a table in shared memory (a row's scale
// times the weight block's), the other warps are the epilogue.
//
// Work: the units are (tile, K block), tile after tile.  A cluster takes a
// contiguous share of whole tiles and its blocks even, contiguous shares of
// the cluster's units, so a block has whole tiles, which it stores, and a part
// of its first and last tile.  Those parts are joined through distributed
// shared memory once, at the end, in the blocks' order: no scratch, and the
// same result every time.
#include <atomic>
#include <type_traits>

#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "stream.cuh"

namespace effort {

struct TcArgs {
  TileMat w;
  const float* ws;  // [out block][K block], rows of nkb4
  int nkb4, O;
  long long rows;
  const float* xs;
  long long xsstride;
  void* out;
  long long ostride;
  int odt, ots, tiles, cluster;  // ots: tiles along the output columns
  WaitHook hook;
};

constexpr int kTurn = 32 * 64;  // 64 bytes of 32 rows
// ROWS: x on the M side.
template <bool ROWS, int M, int N>
struct TcShape {
  static constexpr int kABytes = M * 128, kBBytes = N * 128;
  static constexpr int kTileRows = ROWS ? M : N, kTileCols = ROWS ? N : M;  // of the output
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kEpiWarps = ROWS ? 8 : 4;
  static constexpr int kThreads = (3 + kEpiWarps) * 32 + 32;  // warp 3 is idle: the epilogue starts at a multiple of 4
  // Accumulators in tensor memory, and the steps a K block is multiplied in: 256
  // columns go in two, so that four accumulators fit and the epilogue has three
  // steps' time to read one (with two of 256 columns the products waited for it).
  static constexpr int kSteps = N == 256 ? 2 : 1, kStepN = N / kSteps;
  static constexpr int kAcc = kStepN == 128 ? 4 : 8;
  static constexpr int kTmemCols = kAcc * kStepN;
  static constexpr int kSets = kEpiWarps / 4, kCols = kStepN / kSets;  // of one epilogue thread in one step
  static constexpr int kBatch = 8, kBatches = N == 256 ? 2 : 3;  // K blocks whose scales are turned at once
  static constexpr bool kJoins = N <= 128;
  static constexpr int kHead = 1024, kBlocksAt = kHead - 9 * 8;
  // the table of scales of one K block: for ROWS each row's for the 128 columns
  // of each half, else each row's
  static constexpr int kScales = ROWS ? M * (N / 128) : N;
  static constexpr int kScaleBytes = kBatches * kBatch * kScales * 4;
  // a part in shared memory: rows of the output, their columns together (the
  // blocks of a cluster read it 16 bytes a lane); + 4 floats for the banks
  static constexpr int kPitch = kTileCols + 4;
  static constexpr int kPart = kTileRows * kPitch * 4, kJoinBytes = kJoins ? kPart : 0;
  static constexpr int kTurnBytes = ROWS ? kEpiWarps * kTurn : 0;  // where a warp turns its rows to whole sectors
  static constexpr int kFree = kSmemMax - kHead - kScaleBytes - kJoinBytes - kTurnBytes;
  static constexpr int kStages = kFree / kStage > 12 ? 12 : kFree / kStage;
  static constexpr int kScaleAt = kHead + kStages * kStage, kJoinAt = kScaleAt + kScaleBytes,
                       kTurnAt = kJoinAt + kJoinBytes;
  static constexpr size_t kSmem = kTurnAt + kTurnBytes;
  // in the head: the barriers, where tensor memory starts, and whether a wait ran out
  static constexpr int kTmemAt = 8 * (2 * kStages + 2 * kAcc + 2 * kBatches + 1), kBadAt = kTmemAt + 8;
  static_assert(kBadAt + 8 <= kBlocksAt, "the head");
  // parts to join: the first tile's has its own place, the last tile's is
  // written when every stage has been used and lies over them
  __host__ __device__ static constexpr int part(int slot) { return slot == 0 ? kJoinAt : kHead; }
  static_assert(kStages >= 3 && (!kJoins || kPart <= kStages * kStage) && kSmem <= kSmemMax && kTmemCols <= 512, "fits");
};

// a descriptor of a K-major operand tile in the 128-byte swizzle, 8-row groups 1 KB apart
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3ffff) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// One lane of a warp issues, but the whole warp runs the loop around it: the
// instruction takes its operands from uniform registers, which a loop of one
// lane would have to move there one by one.
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
  return e;
}
// ADD: to what the accumulator holds
template <bool ADD>
__device__ __forceinline__ void mma_f8(uint32_t e, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{ .reg .pred p, q; setp.ne.b32 q, %5, 0; setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "n"(ADD ? 1 : 0), "r"(e)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t e, uint32_t bar) {
  asm volatile(
      "{ .reg .pred q; setp.ne.b32 q, %1, 0;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(e)
      : "memory");
}
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tensor_load2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// A wait that gives up at once after this thread's first failure.  The copying,
// matrix and scale warps set *bad before they go on, so that the epilogue stores
// no tile as good from then on; its own failures it knows.  (A store in this
// function instead cost 5%: 307 against 293 us at 4096 x 4096 x 14336.)
__device__ __forceinline__ void tc_wait(const TcArgs& a, uint32_t bar, uint32_t parity, bool& fine) {
  if (fine) fine = mbar_wait(bar, parity, a.hook.tries);
}

// One thread's accumulators to the output: for ROWS C columns of one row, else
// one column of C rows.
template <bool ROWS, int C>
__device__ __forceinline__ void store_tile(const TcArgs& a, const float (&acc)[C], long long r0, int c0, uint4* turn) {
  auto put = [&](auto* o) {
    using T = std::remove_pointer_t<decltype(o)>;
    if constexpr (ROWS) {
      // A lane holds one row, and rows lie far apart: 64 bytes of the warp's 32
      // rows at a time go through shared memory, so that four lanes write 64
      // bytes of a row (16 bytes at a time from each lane alone were half
      // sectors: 60 of 386 us at 4096 x 4096 x 14336), or, where rows do not
      // start on 16 bytes or the tile ends inside them, neighbouring lanes
      // neighbouring elements (each lane its own row: 50 against 15 us at
      // 258 x 1717 x 7342 bf16).
      constexpr int V = 16 / sizeof(T), P = 64 / sizeof(T);  // elements of 16 and of 64 bytes
      const int lane = threadIdx.x & 31, live = a.O - c0;
      const bool aligned = (((uintptr_t)(o + c0) | (uintptr_t)(a.ostride * sizeof(T))) & 15) == 0;
      T* p = o + (r0 - lane) * a.ostride + c0;  // the warp's first row
      const int rows = (int)min(32ll, a.rows - (r0 - lane));
#pragma unroll
      for (int j = 0; j < C; j += P) {
        if (j >= live) break;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          alignas(16) T v[V];
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = from_float<T>(acc[j + q * V + i]);
          turn[lane * 4 + (q ^ ((lane >> 1) & 3))] = *reinterpret_cast<const uint4*>(v);
        }
        __syncwarp();
        if (aligned && live - j >= P) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), q = lane & 3;
            if (r < rows) *reinterpret_cast<uint4*>(p + r * a.ostride + j + q * V) = turn[r * 4 + (q ^ ((r >> 1) & 3))];
          }
        } else {
          const int e = lane % P;
#pragma unroll 4
          for (int r = lane / P; r < rows; r += 32 / P)
            if (j + e < live)
              p[r * a.ostride + j + e] = reinterpret_cast<const T*>(turn + r * 4 + (e / V ^ ((r >> 1) & 3)))[e % V];
        }
      }
    } else {
      if (c0 >= a.O) return;
      T* p = o + r0 * a.ostride + c0;
      const int live = (int)min((long long)C, a.rows - r0);
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j < live) p[j * a.ostride] = from_float<T>(acc[j]);
    }
  };
  if (a.odt == kF32) put((float*)a.out);
  else if (a.odt == kF16) put((__half*)a.out);
  else put((__nv_bfloat16*)a.out);
}

// Four neighbouring outputs, or the first `live` of them.
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 s, int live) {
  alignas(16) const T v[4] = {from_float<T>(s.x), from_float<T>(s.y), from_float<T>(s.z), from_float<T>(s.w)};
  using Wide = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
  if (live >= 4 && ((uintptr_t)p & (sizeof(Wide) - 1)) == 0) *reinterpret_cast<Wide*>(p) = *reinterpret_cast<const Wide*>(v);
  else
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < live) p[i] = v[i];
}

// Steps through a block's units without a division each.
struct Walk {
  int kb, ot, tt;  // K block, output-column tile, row tile
  __device__ Walk(int tile, int kb_, int ots) : kb(kb_), ot(tile % ots), tt(tile / ots) {}
  __device__ void step(int nkb, int ots) {
    if (++kb == nkb) {
      kb = 0;
      if (++ot == ots) {
        ot = 0;
        ++tt;
      }
    }
  }
};

template <bool ROWS, int M, int N>
__global__ void __launch_bounds__(TcShape<ROWS, M, N>::kThreads, 1)
    k_fp8_tc(const __grid_constant__ CUtensorMap xmap, const TcArgs a) {
  using S = TcShape<ROWS, M, N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int cl = a.cluster, rank = cluster_rank();
  const int ncl = gridDim.x / cl, c = blockIdx.x / cl;
  const int T0 = (int)((long long)a.tiles * c / ncl), T1 = (int)((long long)a.tiles * (c + 1) / ncl);
  const int nkb = a.w.nkb;
  // where each block of the cluster starts: its tile (from T0 on) and K block
  const long long units = (long long)(T1 - T0) * nkb;
  const long long u0 = units * rank / cl, u1 = units * (rank + 1) / cl;
  const int mine = (int)(u1 - u0);
  const Walk start(T0 + (int)(u0 / nkb), (int)(u0 % nkb), a.ots);

  // barriers: stage full / free, accumulator full / read, scales full / read
  const uint32_t b_full = sbase, b_free = b_full + 8 * S::kStages, b_accf = b_free + 8 * S::kStages,
                 b_acce = b_accf + 8 * S::kAcc, b_scf = b_acce + 8 * S::kAcc, b_sce = b_scf + 8 * S::kBatches,
                 b_end = b_sce + 8 * S::kBatches;  // b_end: all products done, after a failure
  volatile int* bad = reinterpret_cast<volatile int*>(smem + S::kBadAt);
  int2* from = reinterpret_cast<int2*>(smem + S::kBlocksAt);
  if (threadIdx.x >= 32 && threadIdx.x <= 32 + cl) {
    const long long u = units * (threadIdx.x - 32) / cl;
    from[threadIdx.x - 32] = make_int2((int)(u / nkb), (int)(u % nkb));
  }
  if (threadIdx.x == 0) {
    mbar_init(b_end, 1);
    asm volatile("prefetch.tensormap [%0];" ::"l"(&xmap) : "memory");
    *bad = 0;
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(b_full + 8 * i, 1);
      mbar_init(b_free + 8 * i, 1);
    }
    for (int i = 0; i < S::kAcc; ++i) {
      mbar_init(b_accf + 8 * i, 1);
      mbar_init(b_acce + 8 * i, S::kEpiWarps);
    }
    for (int i = 0; i < S::kBatches; ++i) {
      mbar_init(b_scf + 8 * i, 1);
      mbar_init(b_sce + 8 * i, S::kEpiWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + S::kTmemAt), "n"(S::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + S::kTmemAt);
  bool fine = true;
  int asked = 0;  // stages the copying lane has asked for
  // the widest shape: 384 threads launched with 168 registers; 8 x 32 x 208 + 4 x
  // 32 x 80 fit in them
  if constexpr (N == 256) {
    static_assert(256 * 208 + 128 * 80 <= 384 * 168, "within the block's registers");
  }

  if (warp < 4) {
  if constexpr (N == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  if (warp == 0 && lane == 0) {
    // ------------------------------------------------ copies
    // (one lane: the copies take their operands from the warp's uniform registers)
    const int last_group = a.w.cores / kGroupCores - 1;  // columns behind it are not stored: any weights do
    auto load_w = [&](const Walk& w, int s) {
      mbar_expect(b_full + 8 * s, S::kStage + a.hook.lost(asked++));
#pragma unroll
      for (int h = 0; h < S::kTileCols / 64; ++h)
        bulk_load(sbase + S::kHead + s * S::kStage + (ROWS ? S::kABytes : 0) + h * kGroupBytes,
                  a.w.data + core_at(min(w.ot * (S::kTileCols / 64) + h, last_group) * kGroupCores, w.kb, nkb), kGroupBytes,
                  b_full + 8 * s);
    };
    auto load_x = [&](const Walk& w, int s) {
      tensor_load2(sbase + S::kHead + s * S::kStage + (ROWS ? 0 : S::kABytes), &xmap, w.kb * kBlk, w.tt * S::kTileRows,
                   b_full + 8 * s);
    };
    // the first stages' weights do not depend on the kernel before
    const int early = min(S::kStages, mine);
    Walk w = start, x = start;
    for (int i = 0; i < early; ++i, w.step(nkb, a.ots)) load_w(w, i);
    grid_dep_wait();
    for (int i = 0; i < early; ++i, x.step(nkb, a.ots)) load_x(x, i);
    int s = 0, ph = 0;
    if (early == S::kStages)
      for (int n = early; n < mine; ++n, w.step(nkb, a.ots)) {
        tc_wait(a, b_free + 8 * s, ph, fine);
        if (!fine) {  // the stage may still be read, or not have come
          *bad = 1;
          break;
        }
        load_w(w, s);
        load_x(w, s);
        if (++s == S::kStages) s = 0, ph ^= 1;
      }
  } else if (warp == 1) {
    // ------------------------------------------------ matrix instructions
    grid_dep_wait();  // or the waits below would count the time of the kernel before
    // fp32 sums, e4m3 operands, both K-major, N and M
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(S::kStepN >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
    const uint64_t a0 = smem_desc(sbase + S::kHead);
    const uint32_t e = elect();
    uint32_t frees = e;  // whether this lane hands stages back: none after a failure, so no copy meets another
    int s = 0, ph = 0, as = 0, aph = 1;  // aph: an accumulator's first use waits for nothing
    for (int n = 0; n < mine; ++n) {
      // the stage and the K block's accumulators (kAcc is a multiple of kSteps)
      const uint32_t f = b_full + 8 * s, r = b_acce + 8 * as;
      bool ready;
      if constexpr (S::kSteps == 2) ready = mbar_try3(f, ph, r, aph, r + 8, aph);
      else ready = mbar_try2(f, ph, r, aph);
      if (!ready) {
        tc_wait(a, f, ph, fine);
#pragma unroll
        for (int h = 0; h < S::kSteps; ++h) tc_wait(a, r + 8 * h, aph, fine);
        if (!fine) {
          *bad = 1;
          frees = 0;
        }
      }
      tc_after();
      const uint64_t da = a0 + (uint64_t)(s * (S::kStage >> 4)), db = da + (S::kABytes >> 4);
#pragma unroll
      for (int h = 0; h < S::kSteps; ++h) {
        const uint64_t dh = db + (uint64_t)(h * S::kStepN * 128 >> 4);
        const uint32_t d = tmem + (as + h) * S::kStepN;
        mma_f8<false>(e, d, da, dh, idesc);
#pragma unroll
        for (int k = 1; k < 4; ++k) mma_f8<true>(e, d, da + 2 * k, dh + 2 * k, idesc);
        mma_commit(e, b_accf + 8 * (as + h));
      }
      mma_commit(frees, b_free + 8 * s);
      as += S::kSteps;
      if (as == S::kAcc) as = 0, aph ^= 1;
      if (++s == S::kStages) s = 0, ph ^= 1;
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------ scales
    grid_dep_launch();
    grid_dep_wait();
    constexpr int R = (S::kTileRows + 31) / 32, H = S::kScales / S::kTileRows;  // rows of a lane, halves
    const bool vec = ((uintptr_t)a.xs & 15) == 0 && (a.xsstride & 3) == 0;
    int batch = 0;
    Walk at = start;
    for (int u = 0; u < mine; ++batch) {
      const int kb = at.kb, n = min(min(S::kBatch, nkb - kb), mine - u), sl = batch % S::kBatches;
      float v[R][S::kBatch], w[H][S::kBatch];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        // a tile's last half may lie behind the last block of columns
        const float* pw = a.ws + (size_t)min(at.ot * S::kTileCols / kBlk + h, (a.O - 1) / kBlk) * a.nkb4 + kb;
#pragma unroll
        for (int k = 0; k < S::kBatch; ++k) w[h][k] = k < n ? __ldg(pw + k) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const long long r = (long long)at.tt * S::kTileRows + 32 * i + lane;
        const bool there = 32 * i + lane < S::kTileRows && r < a.rows;
        // plain loads: the kernel before may still have been writing when this one started
        const float* p = a.xs + (there ? r : 0) * a.xsstride + kb;
        if (vec && (kb & 3) == 0 && n == S::kBatch) {
#pragma unroll
          for (int k = 0; k < S::kBatch; k += 4) {
            const float4 q = there ? *reinterpret_cast<const float4*>(p + k) : make_float4(0, 0, 0, 0);
            v[i][k] = q.x, v[i][k + 1] = q.y, v[i][k + 2] = q.z, v[i][k + 3] = q.w;
          }
        } else {
#pragma unroll
          for (int k = 0; k < S::kBatch; ++k) v[i][k] = there && k < n ? p[k] : 0.0f;
        }
      }
      if (batch >= S::kBatches) tc_wait(a, b_sce + 8 * sl, (batch / S::kBatches - 1) & 1, fine);
      if (!fine) *bad = 1;
      float* t = reinterpret_cast<float*>(smem + S::kScaleAt) + sl * S::kBatch * S::kScales;
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < S::kBatch; ++k)
#pragma unroll
          for (int h = 0; h < H; ++h)
            if (32 * i + lane < S::kTileRows) t[k * S::kScales + h * S::kTileRows + 32 * i + lane] = v[i][k] * w[h][k];
      __syncwarp();
      if (lane == 0) mbar_arrive(b_scf + 8 * sl);
      u += n;
      at.kb += n - 1;
      at.step(nkb, a.ots);
    }
  }
  } else {
    // ------------------------------------------------ epilogue
    if constexpr (N == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    grid_dep_wait();  // as above
    const int quarter = warp & 3, set = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;  // lane of tensor memory
    const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + set * S::kCols;
    float acc[S::kSteps][S::kCols];
    int slot = 0, sph = 0;  // batch of scales in use
    Walk w = start;
    bool first_tile = true;
    int as = 0, aph = 0;
    // The columns go in pieces, and the next piece is on its way (into the other
    // half of v) while one is added, over the ends of steps and K blocks too.
    constexpr int kPiece = S::kCols < 32 || N == 256 ? 16 : 32, kPieces = S::kCols / kPiece, kLoads = kPiece / 16;
    static_assert(kPieces == 1 || kPieces % 2 == 0, "a step starts in the first half");
    float v[2][kLoads][16];
    auto open = [&]() {  // the next accumulator's first piece
      tc_wait(a, b_accf + 8 * as, aph, fine);
      tc_after();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) tmem_load16(tm + as * S::kStepN + 16 * i, v[kPieces == 1][i]);
    };
    if (mine > 0) open();
    for (int n = 0; n < mine;) {
      // the rest of a tile, as far as it is this block's; its scales batch by batch
      const int kb_first = w.kb, seg = min(nkb - kb_first, mine - n);
#pragma unroll
      for (int h = 0; h < S::kSteps; ++h)
#pragma unroll
        for (int j = 0; j < S::kCols; ++j) acc[h][j] = 0.0f;
      for (int b0 = 0; b0 < seg; b0 += S::kBatch) {
        const int bn = min(S::kBatch, seg - b0);
        tc_wait(a, b_scf + 8 * slot, sph, fine);
        uint32_t sc = sbase + S::kScaleAt + slot * S::kBatch * S::kScales * 4 + (ROWS ? row * 4 : 0);
        for (int i = 0; i < bn; ++i, sc += S::kScales * 4) {
          const bool more = n + b0 + i + 1 < mine;
#pragma unroll
          for (int h = 0; h < S::kSteps; ++h) {
            float one = 0.0f;                // ROWS: the row's scale
            uint4 f[ROWS ? 1 : kPiece / 4];  // else: a piece's, one for each column
            if constexpr (ROWS) one = lds_float(sc + h * M * 4);
#pragma unroll
            for (int pc = 0; pc < kPieces; ++pc) {
              if constexpr (!ROWS) {
#pragma unroll
                for (int j = 0; j < kPiece / 4; ++j) f[j] = lds128(sc + 4 * pc * kPiece + 16 * j);
              }
              tmem_wait();
              if constexpr (kPieces == 1) {
#pragma unroll
                for (int l = 0; l < kLoads; ++l)
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[0][l][j] = v[1][l][j];
              }
              if (pc + 1 == kPieces) {
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_acce + 8 * as);  // it may be written again
                as = as + 1 == S::kAcc ? 0 : as + 1;
                aph ^= as == 0;
                if (h + 1 < S::kSteps || more) open();
              } else {
#pragma unroll
                for (int l = 0; l < kLoads; ++l)
                  tmem_load16(tm + as * S::kStepN + (pc + 1) * kPiece + 16 * l, v[(pc + 1) & 1][l]);
              }
#pragma unroll
              for (int j = 0; j < kPiece; j += 4) {
                const uint4 g = ROWS ? make_uint4(0, 0, 0, 0) : f[ROWS ? 0 : j / 4];
                float* d = acc[h] + pc * kPiece + j;
                const float* x = &v[pc & 1][j / 16][j % 16];
                d[0] = fmaf(x[0], ROWS ? one : __uint_as_float(g.x), d[0]);
                d[1] = fmaf(x[1], ROWS ? one : __uint_as_float(g.y), d[1]);
                d[2] = fmaf(x[2], ROWS ? one : __uint_as_float(g.z), d[2]);
                d[3] = fmaf(x[3], ROWS ? one : __uint_as_float(g.w), d[3]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_sce + 8 * slot);
        slot = slot + 1 == S::kBatches ? 0 : slot + 1;
        sph ^= slot == 0;
      }
      {
        const float poison = !fine || *bad ? __int_as_float(0x7fffffff) : 0.0f;
        const bool whole = seg == nkb;
        float* part = reinterpret_cast<float*>(smem + S::part(first_tile ? 0 : 1));
#pragma unroll
        for (int h = 0; h < S::kSteps; ++h) {
          const int c0 = h * S::kStepN + set * S::kCols;  // first N-side column of this thread
#pragma unroll
          for (int j = 0; j < S::kCols; ++j) acc[h][j] += poison;
          if (whole)
            store_tile<ROWS, S::kCols>(a, acc[h], (long long)w.tt * S::kTileRows + (ROWS ? row : c0),
                                       w.ot * S::kTileCols + (ROWS ? c0 : row),
                                       reinterpret_cast<uint4*>(smem + S::kTurnAt + (ROWS ? (warp - 4) * kTurn : 0)));
          else if (S::kJoins) {
            if constexpr (ROWS) {
#pragma unroll
              for (int j = 0; j < S::kCols; j += 4)
                *reinterpret_cast<float4*>(part + row * S::kPitch + c0 + j) =
                    make_float4(acc[h][j], acc[h][j + 1], acc[h][j + 2], acc[h][j + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < S::kCols; ++j) part[(c0 + j) * S::kPitch + row] = acc[h][j];
            }
          }
        }
        first_tile = false;
      }
      n += seg;
      w.kb += seg - 1;
      w.step(nkb, a.ots);
    }
  }
  if (!fine) *bad = 1;
  __syncwarp();
  if (warp != 2) grid_dep_launch();
  tc_before();
  __syncthreads();
  const bool failed = *bad;  // the same in every thread
  if (failed) {
    // copies and products in flight end before the block does (as long as a wait
    // lasts), and its parts say that they are none
    if (threadIdx.x == 0)
      for (int i = max(0, asked - S::kStages); i < asked && mbar_wait(b_full + 8 * (i % S::kStages), i / S::kStages & 1, a.hook.tries);) ++i;
    if (warp == 1) {
      mma_commit(elect(), b_end);
      mbar_wait(b_end, 0, a.hook.tries);
    }
    __syncthreads();
    if constexpr (S::kJoins)
      for (int i = threadIdx.x; i < S::kPart / 4; i += S::kThreads)
        for (int slot = 0; slot < 2; ++slot) reinterpret_cast<float*>(smem + S::part(slot))[i] = __int_as_float(0x7fffffff);
  }
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmemCols));
  if (!S::kJoins || cl == 1) return;
  cluster_sync();
  for (int i = 1; i < cl; ++i) {
    // the tile that block i starts in the middle of, if it is the first to
    const int t = from[i].x;
    if (from[i].y == 0 || (from[i - 1].x == t && from[i - 1].y != 0)) continue;
    int last = i;  // blocks i - 1 .. last have a part of it
    while (last + 1 < cl && from[last + 1].x == t) ++last;
    const int tile = T0 + t, ot = tile % a.ots, tt = tile / a.ots;
    // neighbouring threads take neighbouring output columns
    const int live = (int)min((long long)S::kTileRows, a.rows - (long long)tt * S::kTileRows);
    constexpr int Q = S::kTileCols / 4;
    for (int e = rank * (int)blockDim.x + threadIdx.x; e < live * Q; e += cl * (int)blockDim.x) {
      const int r = e / Q, o = e % Q * 4, col = ot * S::kTileCols + o;
      const uint32_t at = (uint32_t)(r * S::kPitch + o) * 4;
      float4 s = make_float4(0, 0, 0, 0);
      for (int b = i - 1; b <= last; ++b) {
        const float4 p = remote_float4(sbase + S::part(from[b].x == t ? 0 : 1) + at, b);
        s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
      }
      const size_t to = ((long long)tt * S::kTileRows + r) * a.ostride + col;
      if (a.odt == kF32) store4(static_cast<float*>(a.out) + to, s, a.O - col);
      else if (a.odt == kF16) store4(static_cast<__half*>(a.out) + to, s, a.O - col);
      else store4(static_cast<__nv_bfloat16*>(a.out) + to, s, a.O - col);
    }
  }
  cluster_sync();  // no block leaves while its parts are read
}

// ---------------------------------------------------------------- host
template <bool ROWS, int M, int N>
static cudaError_t launch_tc(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                             const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                             cudaStream_t s) {
  using S = TcShape<ROWS, M, N>;
  static std::atomic<int> fit[kMaxDevices][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cfg.attrs = at;
  if (fit[dev][0].load() == 0) {
    e = cudaFuncSetAttribute(k_fp8_tc<ROWS, M, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess) return e;
    for (int i = 3; i >= 0; --i) {
      at[0].val.clusterDim.x = 1u << i;
      cfg.gridDim = dim3(1u << i);
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, k_fp8_tc<ROWS, M, N>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      fit[dev][i].store(n);
    }
    if (fit[dev][0].load() < 1) return cudaErrorLaunchOutOfResources;
  }
  const int ots = cdiv(O, S::kTileCols), nkb = w.nkb;
  const long long tiles = (long long)ots * cdiv(rows, S::kTileRows);
  if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
  TcArgs a = {w, ws, align4(nkb), O, rows, xs, xsstride, out, ostride, odt, ots, (int)tiles, 1, wait_hook()};
  // the cluster size whose longest share of units is shortest; the join is
  // counted as eight of them
  long long best = 0;
  int ncl = 0;
  for (int i = 0; i < (S::kJoins ? 4 : 1); ++i) {
    const long long cl = 1ll << i, n = fit[dev][i].load() < tiles ? fit[dev][i].load() : tiles;
    if (n < 1 || cl > nkb) break;
    const long long per = (tiles + n - 1) / n * nkb, cost = (per + cl - 1) / cl + (cl > 1 ? 8 : 0);
    if (ncl == 0 || cost < best) {
      best = cost;
      a.cluster = (int)cl;
      ncl = (int)n;
    }
  }
  CUtensorMap xmap;
  if (!map_rows(&xmap, x, I, rows, xstride, S::kTileRows)) return cudaErrorInvalidValue;
  at[0].val.clusterDim.x = (unsigned)a.cluster;
  cfg.gridDim = dim3((unsigned)(ncl * a.cluster));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_fp8_tc<ROWS, M, N>, xmap, a);
}

cudaError_t launch_fp8_tc(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                          const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                          cudaStream_t s) {
#define GO(ROWS, M, N) return launch_tc<ROWS, M, N>(w, ws, I, O, x, xstride, xs, xsstride, rows, odt, out, ostride, s)
  if (rows <= 16) GO(false, 128, 16);
  if (rows <= 32) GO(false, 128, 32);
  if (rows <= 64) GO(false, 128, 64);
  // Tiles of 128 x 128 split their K over a cluster where they are few; 128 x 256
  // reads less and adds more at once, but goes in whole tiles, 148 at a time.
  // Measured, 128 x 128 / 128 x 256 in us, by tiles of 128 x 256:
  //   tiles       16        64         80         112        168        224        280        448        512
  //   K = 4096    11.0/23.7 18.7/26.0  29.0/27.1  31.8/28.9  42.5/49.4  54.4/49.5  57.4/51.5  90.7/91.8  93.5/90.8
  //   K = 1024    5.8/9.0   7.2/9.4    11.2/10.5  11.1/11.1  14.6/19.4  17.8/19.1  19.8/21.4  30.0/35.6  30.2/35.6
  // From 149 tiles on, just behind a whole round, the wide shape is up to a third
  // slower, and at a short K up to a fifth throughout; the rule does not see that.
  if ((long long)cdiv(O, 256) * cdiv(rows, 128) < 100) GO(true, 128, 128);
  GO(true, 128, 256);
#undef GO
}

}  // namespace effort
