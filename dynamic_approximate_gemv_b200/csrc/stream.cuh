// Products with few columns: device code shared by the e4m3 product (fp8.cu)
// and the mixture of experts (moe.cu).
//
// What bounds them is the one read of the weights, so the kernel is built
// around that stream.  One block per SM.  A block works through groups of up
// to MT 16-row tiles; inside a group warp w multiplies the K blocks w, w + kw,
// ...  Each warp owns a ring of stages in shared memory that it fills itself
// with bulk copies and runs ahead through its whole list, across the groups'
// borders, so no warp waits for another except in the join at a group's end.
//
// A stage brings everything one K block of a group needs: the weights' cores
// (1 KB each), that K block of the activations' rows, and its scales, so no
// warp waits for L2 between two stages (loads of the activations in the loop
// cost 14.9 against 11.1 us without them at 1 x 4096 x 14336).
//
// The products run on the warp-wide matrix instruction m16n8k16 (16 weight
// rows, 8 columns, fp32 sums): with so few columns every operand byte is used
// once and the larger instructions would wait for HBM just the same.  e4m3
// weights become binary16 in registers (exact).  K may be permuted freely as
// long as both operands agree: lane q of a row's four takes 32 consecutive
// bytes, which are two 16-byte reads that meet no bank twice.
#pragma once
#include <stdlib.h>

#include "ffn_common.cuh"

namespace effort {

constexpr int kMaxWaits = 1 << 18;  // tries of a wait before it gives up

// The debug build lets a test make waits run out: EFFORT_TEST_WAIT_TRIES is the
// number of tries, and with EFFORT_TEST_LOST_COPY=n the n-th and later stages of a
// ring wait for 16 bytes that no copy brings.
#ifdef EFFORT_DEBUG
struct WaitHook {
  int tries = kMaxWaits, after = 0x7fffffff;
  __host__ __device__ int lost(int n) const { return n >= after ? 16 : 0; }
};
inline WaitHook wait_hook() {
  WaitHook h;
  if (const char* t = getenv("EFFORT_TEST_WAIT_TRIES")) h.tries = atoi(t);
  if (const char* t = getenv("EFFORT_TEST_LOST_COPY")) h.after = atoi(t);
  return h;
}
#else
struct WaitHook {
  static constexpr int tries = kMaxWaits;
  __host__ __device__ static constexpr int lost(int) { return 0; }
};
inline WaitHook wait_hook() { return {}; }
#endif

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded: false once the phase did not come.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, int tries) {
  for (int i = 0; i < tries; ++i)
    if (mbar_try(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int tries = kMaxWaits) {
  return mbar_try(bar, parity) || mbar_wait_long(bar, parity, tries);
}
// A ready barrier takes 129 clocks to say so (B200, one warp), but several asked
// together take no longer: whether all are in their phases.
__device__ __forceinline__ bool mbar_try2(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p, q; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4; and.pred p, p, q; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_try3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p, q, r; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 r, [%5], %6;\n"
      "and.pred p, p, q; and.pred p, p, r; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2)
      : "memory");
  return ok != 0;
}
// both addresses and the size are multiples of 16 bytes
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// The barrier of one set of `warps` warps out of a block's; at most 8 sets of two
// warps or more.  (Not barrier 0: that is the whole block's, and a set that has
// gone on to the block's barrier must not meet another still at its own.)
__device__ __forceinline__ void set_sync(int set, int warps) {
  if (warps == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(set + 1), "r"(warps * 32) : "memory");
}
// The warp's number and the block's rank in its cluster, through a shuffle, by
// which the compiler knows that they are the same in every lane: branches on
// them, and all that is computed from them, then need no convergence barriers
// (a K block of the epilogue spent 500 of 750 clocks in those).
__device__ __forceinline__ int warp_index() { return __shfl_sync(~0u, (int)(threadIdx.x >> 5), 0); }
__device__ __forceinline__ int cluster_rank() {
  int r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return __shfl_sync(~0u, r, 0);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float remote_float(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_float4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_float(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two fp32 values to a pair of the matrix instruction's type, low half first
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (BF16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
// four e4m3 values as two pairs of binary16
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
      : "=r"(a), "=r"(b)
      : "r"(w));
}

// Power of two that brings a block's largest magnitude into [2^14, 2^15), the
// top of binary16's range, and its inverse.  Blocks below 2^-97 are scaled as
// if they reached it.
__device__ __forceinline__ void pow2_scale(float amax, float* up, float* down) {
  int e = (int)((__float_as_uint(amax) >> 23) & 0xff);  // biased exponent; inf and NaN: 255
  e = e < 30 ? 30 : e;
  *up = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
  *down = __uint_as_float((uint32_t)(e - 14) << 23);
}

// ---------------------------------------------------------------- shapes
// What a stage holds and how many fit: W warps, MT tiles a group, ST stages a
// warp.  ROWS: activation rows, ROWB: bytes of one K block of a row, PAD: bytes
// between rows (with it no read of the fragments meets a bank twice), EXTRA:
// shared memory of the caller's own.
constexpr int kSmemMax = 227 * 1024;
constexpr int kStreamHead = 2048;    // barriers
template <int ROWS, int ROWB, int PAD, int EXTRA>
struct StreamShape {
  static constexpr int NT = (ROWS + 7) / 8;  // column tiles of 8
  static constexpr int kRowPitch = ROWB + PAD;
  static constexpr int kActBytes = ROWS * kRowPitch;
  static constexpr int stage(int mt) { return mt * 2 * kCoreBytes + kActBytes + 64; }
  static constexpr int pitch(int mt) { return mt * 16 + 4; }  // floats of a column in the join, likewise
  static constexpr int red(int w, int mt) { return w * NT * 8 * pitch(mt) * 4; }
  static constexpr int stages(int w, int mt) {
    const int n = (kSmemMax - kStreamHead - EXTRA - red(w, mt)) / (w * stage(mt));
    return n > 6 ? 6 : n;
  }
  // sixteen warps where two stages each fit (a K block's share of latency
  // hides better than with eight: 12.3 against 14.5 us at 14336 x 4096)
  static constexpr int kPick = stages(16, 2) >= 2 ? 0 : stages(8, 4) >= 2 ? 1 : stages(8, 2) >= 2 ? 2 : 3;
  static constexpr int kWarps = kPick == 0 ? 16 : kPick == 3 ? 6 : 8;
  static constexpr int kMT = kPick == 1 ? 4 : 2;
  static constexpr int kStages = stages(kWarps, kMT);
  static_assert(kStages >= 2, "a ring of two stages");
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStage = stage(kMT);
  static constexpr int kScaleAt = kMT * 2 * kCoreBytes + kActBytes;
  static constexpr int kActAt = kMT * 2 * kCoreBytes;
  static constexpr int kPitch = pitch(kMT);
  static constexpr int kRed = NT * 8 * kPitch;  // floats of one warp's part
  static constexpr int kRingAt = kStreamHead;
  static constexpr int kRedAt = kRingAt + kWarps * kStages * kStage;
  static constexpr int kExtraAt = kRedAt + red(kWarps, kMT);
  static constexpr size_t kSmem = kExtraAt + EXTRA;
};

// One warp's ring.  A warp whose wait ran out (fine is false) asks for nothing more;
// its sums are to be poisoned, and drain() lets the copies that are in flight end
// before the block does.  Its lanes vote on each wait, so that they stay together.
template <typename S>
struct Ring {
  uint32_t buf, bar;
  int put = 0, got = 0;  // stages asked for and taken
  bool fine = true;
  __device__ void init(uint32_t sbase, int warp, int lane) {
    buf = sbase + S::kRingAt + warp * S::kStages * S::kStage;
    bar = sbase + warp * S::kStages * 8;
    if (lane < S::kStages) mbar_init(bar + lane * 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
  __device__ uint32_t next_buf() const { return buf + (put % S::kStages) * S::kStage; }
  __device__ uint32_t next_bar() const { return bar + (put % S::kStages) * 8; }
  // the next stage; stop() after a failure sees to it that no more are asked for
  template <typename F>
  __device__ uint32_t wait(uint8_t* smem, int warp, WaitHook hook, F&& stop) {
    const int s = got % S::kStages, parity = (got / S::kStages) & 1;
    if (!__all_sync(~0u, mbar_try(bar + s * 8, parity)) && fine &&
        !__all_sync(~0u, mbar_wait_long(bar + s * 8, parity, hook.tries))) {
      reinterpret_cast<int2*>(smem + kLateAt)[warp] = make_int2(got, put);
      fine = false;
      stop();
    }
    ++got;
    return buf + s * S::kStage;
  }
  __device__ void drain(const uint8_t* smem, int warp, int lane, WaitHook hook) const {
    if (lane != 0 || fine) return;
    const int2 late = reinterpret_cast<const int2*>(smem + kLateAt)[warp];
    for (int i = late.x; i < late.y && mbar_wait(bar + i % S::kStages * 8, (i / S::kStages) & 1, hook.tries); ++i) {}
  }
  // behind the barriers: the stages that each warp had got and asked for when its wait ran out
  static constexpr int kLateAt = S::kWarps * S::kStages * 8;
  static_assert(kLateAt + S::kWarps * 8 <= kStreamHead, "the head");
};

// The second of two binary16 parts is stored times 2^11 (store_parts), and so are its sums.
constexpr float kLowUp = 2048.0f, kLowDown = 1.0f / 2048.0f;

// A fragments of one 16-row tile and K block (two cores in shared memory) times
// the B fragments of NT column tiles, `live` of them in use, added to c.
// k-step s takes the lane's elements 4 s .. 4 s + 3.
template <int WK, int NT, int PARTS, int KS>
__device__ __forceinline__ void mma_tile(uint32_t tile, int g, int q, const uint32_t (&b)[PARTS][NT][KS][2], int live,
                                         float (&c)[NT][4]) {
  const uint32_t r = tile + g * 128;
  const uint32_t c0 = (uint32_t)(((2 * q) ^ g) << 4), c1 = (uint32_t)(((2 * q + 1) ^ g) << 4);
  const uint4 v0 = lds128(r + c0), v1 = lds128(r + c1), v2 = lds128(r + kCoreBytes + c0), v3 = lds128(r + kCoreBytes + c1);
  const uint32_t lo[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  const uint32_t hi[8] = {v2.x, v2.y, v2.z, v2.w, v3.x, v3.y, v3.z, v3.w};
  constexpr bool kLow = PARTS == 2 && WK != kWBF16;
  float low[kLow ? NT : 1][4] = {};
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint32_t a0, a1, a2, a3;
    if constexpr (WK == kWE4M3) {
      e4m3x4_to_half2(lo[s], a0, a2);
      e4m3x4_to_half2(hi[s], a1, a3);
    } else {
      a0 = lo[2 * s];
      a2 = lo[2 * s + 1];
      a1 = hi[2 * s];
      a3 = hi[2 * s + 1];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (NT > 1 && t >= live) break;
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        mma16<WK == kWBF16>(kLow && p == 1 ? low[kLow ? t : 0] : c[t], a0, a1, a2, a3, b[p][t][s][0], b[p][t][s][1]);
    }
  }
  if constexpr (kLow) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[t][e] = fmaf(low[t][e], kLowDown, c[t][e]);
  }
}

// ---------------------------------------------------------------- activations of 16 and 32 bits
// Activations meet 16-bit operands in parts: v = p0 + p1 + .., each of 11
// (binary16) or 8 (bfloat16) significant bits.  For binary16 a K block of a row
// is first scaled by a power of two into its range, and the inverse stands
// behind the parts.  A second binary16 part is scaled by 2^11 once more, so that
// it ends where the first does: with the block's bound at 2^14 or more the parts
// hold 11 and 22 bits of what lies up to 2^28 below the bound, and what lies deeper
// to within 2^-39 and 2^-50 of the bound (with both parts on one scale 22 bits
// ended at 2^-17, and a column of w1 and one of w3 a thousand times the others left
// these 8).  The parts lie in the order of the fragments: of a K block
// of KE elements lane q of a row's four multiplies KE / 4 neighbours, and the
// 16-byte pieces of the four lanes alternate, so that a warp reads 64 bytes of
// a row.
template <int KE>
__host__ __device__ __forceinline__ int frag_pos(int k) {
  constexpr int L = KE / 4;
  const int q = k / L, r = k % L;
  return (r / 8 * 4 + q) * 8 + r % 8;
}
// bytes of one K block of a row
template <int KE, int PARTS, bool SCALED>
__host__ __device__ constexpr int act_block() {
  return KE * 2 * PARTS + (SCALED ? 16 : 0);
}
// v (scaled) into the parts of one element
template <bool BF16, int PARTS>
__device__ __forceinline__ void store_parts(uint16_t* at, int stride, float v) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    if constexpr (BF16) {
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      at[p * stride] = __bfloat16_as_ushort(h);
      v -= __bfloat162float(h);
    } else {
      const __half h = __float2half_rn(v);
      at[p * stride] = __half_as_ushort(h);
      v = (v - __half2float(h)) * kLowUp;
    }
  }
}
// B fragments of one column tile; b: [part][NT][KS][2]
template <int PARTS, int NT, int KS>
__device__ __forceinline__ void act_load(uint32_t row, int q, bool there, uint32_t (&b)[PARTS][NT][KS][2], int j) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p)
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      const uint4 v = there ? lds128(row + p * KS * 32 + (i * 4 + q) * 16) : make_uint4(0, 0, 0, 0);
      b[p][j][2 * i][0] = v.x;
      b[p][j][2 * i][1] = v.y;
      b[p][j][2 * i + 1][0] = v.z;
      b[p][j][2 * i + 1][1] = v.w;
    }
}

// B fragments of one column tile from e4m3 rows in the stage: `left` bytes of
// the K block exist, the rest counts as zero; rows beyond `rows` too.
__device__ __forceinline__ void act_e4m3(uint32_t row, int q, bool there, int left, uint32_t (&b)[8][2]) {
  uint32_t u[8] = {};
  if (there) {
    const uint4 v0 = lds128(row + 32 * q), v1 = lds128(row + 32 * q + 16);
    u[0] = v0.x, u[1] = v0.y, u[2] = v0.z, u[3] = v0.w, u[4] = v1.x, u[5] = v1.y, u[6] = v1.z, u[7] = v1.w;
  }
  if (left < 128) {
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int l = left - (32 * q + 4 * s);
      u[s] &= l >= 4 ? ~0u : l <= 0 ? 0u : (1u << (8 * l)) - 1;
    }
  }
#pragma unroll
  for (int s = 0; s < 8; ++s) e4m3x4_to_half2(u[s], b[s][0], b[s][1]);
}

}  // namespace effort
