// A mixture-of-experts layer for a few tokens:
//
//   l = G x;  ids, gates = top-k of l;  out = sum_j gates_j W2^T (silu(W1^T x) * (W3^T x)),  W of expert ids_j
//
// Four kernels, each started early and waiting for the one before on the
// device: the router (and x in the order the products read it), the first
// products with the gate (w1 and w3 are stored core by core in turn, so a
// matrix instruction's 16 rows are 8 hidden units of both, and a thread has
// both sums of a unit), the second product, and the weighted sum.
//
// The chosen experts' weights are read once each: pairs (token, expert) are
// grouped by expert into chunks of up to 8 or 16 columns, and the 16-row tiles
// of all chunks are dealt to one block per SM in even, contiguous shares of
// the stream described in stream.cuh.  The second product's K is cut into
// shares where its tiles alone would not fill the SMs; the shares' sums are
// added in order.
#include <atomic>

#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "moe.cuh"
#include "stream.cuh"

namespace effort {

// ---------------------------------------------------------------- router
constexpr int kRouterThreads = 512;

// One block per token: x to fragment order, the logits by warps, the top-k by
// one warp.
template <typename T, int KE>
__global__ void __launch_bounds__(kRouterThreads) k_moe_router(const MoeCall c) {
  extern __shared__ float xs[];  // the token, fp32, padded with zeros to rpitch
  __shared__ float logit[EFFORT_MAX_EXPERTS];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = warp_index(), E = c.n_experts;
  grid_dep_launch();
  grid_dep_wait();
  const T* x = static_cast<const T*>(c.x) + t * c.xstride;
  T* to = static_cast<T*>(c.xop) + (size_t)t * c.xpitch;
  for (int k = threadIdx.x; k < c.xpitch; k += kRouterThreads) {
    const T v = k < c.I ? x[k] : from_float<T>(0.0f);
    to[k / KE * KE + frag_pos<T, KE>(k % KE)] = v;
    if (k < c.rpitch) xs[k] = to_float(v);
  }
  // behind a hidden vector's end
  for (int j = 0; j < c.top_k; ++j)
    for (int k = c.F + threadIdx.x; k < c.hpitch; k += kRouterThreads)
      c.h[(size_t)(t * c.top_k + j) * c.hpitch + k / KE * KE + frag_pos<float, KE>(k % KE)] = 0.0f;
  if (c.gate_mode == EFFORT_GATE_GIVEN) return;
  __syncthreads();
  for (int e = warp; e < E; e += kRouterThreads / 32) {
    float s = 0.0f;
    if (c.rdt == kF32) {
      const float4* r = reinterpret_cast<const float4*>(static_cast<const float*>(c.router) + (size_t)e * c.rpitch);
#pragma unroll 4
      for (int k = lane; k < c.rpitch / 4; k += 32) {
        const float4 a = __ldg(r + k), b = reinterpret_cast<const float4*>(xs)[k];
        s += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
      }
    } else {
      const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(c.router) + (size_t)e * c.rpitch);
#pragma unroll 4
      for (int k = lane; k < c.rpitch / 8; k += 32) {
        const uint4 a = __ldg(r + k);
        const float4 b0 = reinterpret_cast<const float4*>(xs)[2 * k], b1 = reinterpret_cast<const float4*>(xs)[2 * k + 1];
        float2 f[4];
        if (c.rdt == kBF16) f[0] = unpack2<true>(a.x), f[1] = unpack2<true>(a.y), f[2] = unpack2<true>(a.z), f[3] = unpack2<true>(a.w);
        else f[0] = unpack2<false>(a.x), f[1] = unpack2<false>(a.y), f[2] = unpack2<false>(a.z), f[3] = unpack2<false>(a.w);
        s += f[0].x * b0.x + f[0].y * b0.y + f[1].x * b0.z + f[1].y * b0.w;
        s += f[2].x * b1.x + f[2].y * b1.y + f[3].x * b1.z + f[3].y * b1.w;
      }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
    if (lane == 0) logit[e] = s;
  }
  __syncthreads();
  if (warp != 0) return;
  // lane l holds the experts l, l + 32, ..; NaN counts as lowest
  constexpr int kPer = EFFORT_MAX_EXPERTS / 32;
  float l[kPer], top = -INFINITY, all = 0.0f, sum = 0.0f, mine = 0.0f;
  bool bad = false;
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = 32 * i + lane;
    l[i] = e < E ? logit[e] : -INFINITY;
    if (e < E) left |= 1u << i;
    bad |= l[i] != l[i];
    if (l[i] != l[i]) l[i] = -INFINITY;
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, m));
  bad = __any_sync(~0u, bad);
  if (c.gate_mode == EFFORT_GATE_TOP_OF_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (left >> i & 1) all += expf(l[i] - top);
#pragma unroll
    for (int m = 16; m; m >>= 1) all += __shfl_xor_sync(~0u, all, m);
  }
  for (int j = 0; j < c.top_k; ++j) {
    float best = -INFINITY;
    int at = 1 << 20;  // the lowest expert among equals
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((left >> i & 1) && (at == 1 << 20 || l[i] > best)) best = l[i], at = 32 * i + lane;
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      const float ob = __shfl_xor_sync(~0u, best, m);
      const int oa = __shfl_xor_sync(~0u, at, m);
      if (oa != 1 << 20 && (at == 1 << 20 || ob > best || (ob == best && oa < at))) best = ob, at = oa;
    }
    if ((at & 31) == lane) left &= ~(1u << (at >> 5));
    const float g = expf(best - top);
    sum += g;
    if (lane == j) {
      mine = g;
      c.ids[t * c.top_k + j] = at;
    }
  }
  const float d = c.gate_mode == EFFORT_GATE_SOFTMAX_OF_TOP ? sum : all;
  if (lane < c.top_k) c.gates[t * c.top_k + lane] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(mine, d);
}

// ---------------------------------------------------------------- the plan
// Pairs by expert, in rising order, cut into chunks of up to `cols`.  Every
// block of a product makes it for itself from the ids.
constexpr int kMaxPairs = EFFORT_MAX_TOKENS * EFFORT_MAX_TOP_K;
struct Plan {
  uint16_t list[kMaxPairs];  // pairs, expert after expert
  uint32_t chunk[EFFORT_MAX_EXPERTS + kMaxPairs / 8];  // start << 13 | count << 8 | expert
  int chunks;
};
static_assert(EFFORT_MAX_EXPERTS <= 256 && kMaxPairs <= 1 << 13, "a chunk's fields");

// temp: 2 kMaxPairs + 4 EFFORT_MAX_EXPERTS bytes
__device__ void make_plan(Plan* p, const int* ids, int pairs, int E, int cols, uint16_t* rank, int* cnt, int warp, int lane,
                          int threads) {
  for (int e = threadIdx.x; e < E; e += threads) cnt[e] = 0;
  __syncthreads();
  if (warp == 0) {
    // a pair's place among those of its expert
    for (int b = 0; b < pairs; b += 32) {
      const int id = b + lane < pairs ? ids[b + lane] : -1;
      const bool ok = id >= 0 && id < E;
      const unsigned same = __match_any_sync(~0u, ok ? id : -1 - lane);
      const int before = __popc(same & ((1u << lane) - 1));
      int base = 0;
      if (ok) base = cnt[id];
      __syncwarp();
      if (ok) {
        rank[b + lane] = (uint16_t)(base + before);
        if (before == 0) cnt[id] = base + __popc(same);
      }
      __syncwarp();
    }
    // starts of the lists and of the chunks, 8 experts a lane
    constexpr int kPer = EFFORT_MAX_EXPERTS / 32;
    int n = 0, m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i, k = e < E ? cnt[e] : 0;
      n += k;
      m += (k + cols - 1) / cols;
    }
    int n0 = n, m0 = m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(~0u, n0, d), b = __shfl_up_sync(~0u, m0, d);
      if (lane >= d) n0 += a, m0 += b;
    }
    if (lane == 31) p->chunks = m0;
    n0 -= n;
    m0 -= m;
    for (int i = 0; i < kPer; ++i) {
      const int e = lane * kPer + i;
      if (e >= E) break;
      const int k = cnt[e];
      for (int s = 0; s < k; s += cols)
        p->chunk[m0++] = (uint32_t)(n0 + s) << 13 | (uint32_t)min(cols, k - s) << 8 | (uint32_t)e;
      cnt[e] = n0;
      n0 += k;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += threads) {
    const int id = ids[i];
    if (id >= 0 && id < E) p->list[cnt[id] + rank[i]] = (uint16_t)i;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- products
template <int WK, typename T, int NT>
using MoeShape = StreamShape<NT, (WK == kWE4M3 ? 128 : 64) * (int)sizeof(T), 64, (int)(sizeof(Plan) + 15) / 16 * 16>;

// DOWN: the second product (T is float).  FEW: see ActKind.
template <int WK, typename T, bool FEW, int NT, bool DOWN>
__global__ void __launch_bounds__(MoeShape<WK, T, NT>::kThreads, 1) k_moe_product(const MoeCall c) {
  using S = MoeShape<WK, T, NT>;
  using A = ActKind<WK, T, FEW>;
  constexpr int MT = S::kMT, W = S::kWarps, KE = WK == kWE4M3 ? 128 : 64, KS = KE / 16, ROWB = KE * (int)sizeof(T);
  // every K block's sums apart, to be scaled, or all into one
  constexpr bool kApart = WK == kWE4M3 || A::kScaled;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float* red = reinterpret_cast<float*>(smem + S::kRedAt);
  Plan* plan = reinterpret_cast<Plan*>(smem + S::kExtraAt);
  const int lane = threadIdx.x & 31, warp = warp_index(), g = lane >> 2, q = lane & 3;
  const TileMat w = DOWN ? c.w2 : c.w13;
  const int nkb = w.nkb, nkb4 = align4(nkb), pairs = c.n_tokens * c.top_k;
  const int tiles = DOWN ? cdiv(c.I, 16) : cdiv(c.F, 8), shares = DOWN ? c.shares : 1;

  grid_dep_launch();
  grid_dep_wait();
  uint8_t* temp = smem + S::kRingAt;  // the ring is not in use yet
  make_plan(plan, c.ids, pairs, c.n_experts, 8 * NT, reinterpret_cast<uint16_t*>(temp),
            reinterpret_cast<int*>(temp + 2 * kMaxPairs), warp, lane, S::kThreads);
  Ring<S> ring;
  ring.init(sbase, warp, lane);
  const int units = plan->chunks * shares * tiles;
  const int u0 = (int)((long long)units * blockIdx.x / gridDim.x), u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);

  // a group: up to MT tiles of one chunk (and K share), inside 64 stored rows
  struct Group {
    int expert, start, count, t, n, kb0, kb1, share;
  };
  auto group_at = [&](int u) {
    Group G;
    const int seg = u / tiles;
    G.t = u - seg * tiles;
    G.share = DOWN ? seg % shares : 0;
    const uint32_t ch = plan->chunk[DOWN ? seg / shares : seg];
    G.expert = ch & 255;
    G.count = ch >> 8 & 31;
    G.start = ch >> 13;
    G.n = min(min(MT, 4 - (G.t & 3)), min(tiles - G.t, u1 - u));
    G.kb0 = DOWN ? nkb * G.share / shares : 0;
    G.kb1 = DOWN ? nkb * (G.share + 1) / shares : nkb;
    return G;
  };
  // what the warp asks for next
  int pu = u0, pk = 0;
  Group P = {};
  auto seek = [&]() {  // the first group from pu on that has a K block for this warp
    while (pu < u1) {
      P = group_at(pu);
      pk = P.kb0 + warp;
      if (pk < P.kb1) return;
      pu += P.n;
    }
  };
  auto ask = [&]() {
    if (pu >= u1) return;
    const uint32_t buf = ring.next_buf(), bar = ring.next_bar();
    constexpr int kScales = WK == kWE4M3 ? (DOWN ? 1 : 2) : 0;
    if (lane == 0) {
      mbar_expect(bar, P.n * 2 * kCoreBytes + P.count * ROWB + 16 * kScales);
      bulk_load(buf, w.data + P.expert * w.stride + core_at(2 * P.t, pk, nkb), P.n * 2 * kCoreBytes, bar);
    }
    __syncwarp();
    if (lane >= 8 && lane - 8 < P.count) {
      const int p = plan->list[P.start + lane - 8];
      const T* row = DOWN ? reinterpret_cast<const T*>(c.h) + (size_t)p * c.hpitch
                          : static_cast<const T*>(c.xop) + (size_t)(p / c.top_k) * c.xpitch;
      bulk_load(buf + S::kActAt + (lane - 8) * S::kRowPitch, row + pk * KE, ROWB, bar);
    }
    if (kScales > 0 && lane >= 1 && lane <= kScales) {
      const float* s = DOWN ? c.s2 : lane == 1 ? c.s1 : c.s3;
      const int nsb = DOWN ? c.nsb2 : c.nsb13, blk = DOWN ? P.t / 8 : P.t / 16;
      bulk_load(buf + S::kScaleAt + 16 * (lane - 1), s + ((size_t)P.expert * nsb + blk) * nkb4 + (pk & ~3), 16, bar);
    }
    ++ring.put;
    pk += W;
    if (pk >= P.kb1) {
      pu += P.n;
      seek();
    }
  };
  seek();
#pragma unroll 1
  for (int s = 0; s < S::kStages; ++s) ask();

  bool fine = true;
  for (int u = u0; u < u1;) {
    const Group G = group_at(u);
    u += G.n;
    const int live = NT == 1 ? 1 : (G.count + 7) / 8;
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    for (int kb = G.kb0 + warp; kb < G.kb1; kb += W) {
      uint32_t at;
      fine &= ring.wait(&at);
      uint32_t b[A::kParts][NT][KS][2];
      float sx[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float down = 1.0f;
        if (j == 0 || j < live)
          act_parts<WK, T, FEW, KS>(at + S::kActAt + (8 * j + g) * S::kRowPitch, q, 8 * j + g < G.count, &b[0][j], NT, &down);
        // the lanes that hold column 2 q (+ 1) know its scale
#pragma unroll
        for (int e = 0; e < 2; ++e) sx[j][e] = A::kScaled ? __shfl_sync(~0u, down, (2 * q + e) * 4) : 1.0f;
      }
      float sw[2] = {1.0f, 1.0f};  // of the tile's rows g and g + 8
      if constexpr (WK == kWE4M3) {
        sw[0] = lds_float(at + S::kScaleAt + 4 * (kb & 3));
        sw[1] = DOWN ? sw[0] : lds_float(at + S::kScaleAt + 16 + 4 * (kb & 3));
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= G.n) break;
        if constexpr (kApart) {
          float d[NT][4] = {};
          mma_tile<WK, NT, A::kParts, KS>(at + m * 2 * kCoreBytes, g, q, b, live, d);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(d[j][e] * sx[j][e & 1], sw[e >> 1], acc[m][j][e]);
        } else {
          mma_tile<WK, NT, A::kParts, KS>(at + m * 2 * kCoreBytes, g, q, b, live, acc[m]);
        }
      }
      __syncwarp();  // every lane has read the stage
      ask();
    }
    // join the warps' sums
    __syncthreads();
    float* mine = red + warp * S::kRed;
    const float poison = fine ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * q + (e & 1)) * S::kPitch + 16 * m + g + 8 * (e >> 1)] = acc[m][j][e] + poison;
    __syncthreads();
    constexpr int kWide = DOWN ? MT * 16 : MT * 8;  // outputs of a column
    for (int i = threadIdx.x; i < G.count * kWide; i += S::kThreads) {
      const int col = i / kWide, o = i % kWide;
      const float* r = red + col * S::kPitch + (DOWN ? o : o / 8 * 16 + o % 8);
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int v = 0; v < W; ++v) {
        a += r[v * S::kRed];
        if (!DOWN) b += r[v * S::kRed + 8];
      }
      const int p = plan->list[G.start + col];
      if constexpr (DOWN) {
        const int row = G.t * 16 + o;
        if (o < G.n * 16 && row < c.I) c.z[((size_t)G.share * pairs + p) * c.I + row] = a;
      } else {
        const int j = G.t * 8 + o;
        if (o < G.n * 8 && j < c.F)
          c.h[(size_t)p * c.hpitch + j / KE * KE + frag_pos<float, KE>(j % KE)] = __fdiv_rn(a, 1.0f + expf(-a)) * b;
      }
    }
  }
}

// out[t] = sum over its pairs and the K shares, in order
__global__ void __launch_bounds__(256) k_moe_sum(const MoeCall c) {
  const int t = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x, pairs = c.n_tokens * c.top_k;
  grid_dep_launch();
  grid_dep_wait();
  if (i >= c.I) return;
  float y = 0.0f;
  for (int j = 0; j < c.top_k; ++j) {
    const int p = t * c.top_k + j, e = c.ids[p];
    if (e < 0 || e >= c.n_experts) continue;
    float a = 0.0f;
    for (int s = 0; s < c.shares; ++s) a += c.z[((size_t)s * pairs + p) * c.I + i];
    y += c.gates[p] * a;
  }
  store_dt(c.out, c.odt, t * c.ostride + i, y);
}

// ---------------------------------------------------------------- host
// every kernel of a call may start before the one ahead of it ends and waits for it itself
template <typename K>
static cudaError_t start(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, const MoeCall& c) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, c);
}
// raises a kernel's shared-memory limit once per device
template <typename K>
static cudaError_t allow(K kernel, std::atomic<bool>* done, size_t smem) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev].load()) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done[dev].store(true);
  return e;
}

template <int WK, typename T, bool FEW, int NT, bool DOWN>
static cudaError_t product(const MoeCall& c, int sms, cudaStream_t s) {
  using S = MoeShape<WK, T, NT>;
  static_assert(S::kWarps * S::kStages * S::kStage >= 2 * kMaxPairs + 4 * EFFORT_MAX_EXPERTS, "the plan's working space");
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow(k_moe_product<WK, T, FEW, NT, DOWN>, done, S::kSmem);
  if (e != cudaSuccess) return e;
  return start(k_moe_product<WK, T, FEW, NT, DOWN>, dim3((unsigned)sms), S::kThreads, S::kSmem, s, c);
}
template <int WK, typename T>
static cudaError_t up(const MoeCall& c, int sms, cudaStream_t s) {
  return c.n_tokens <= 8 ? product<WK, T, false, 1, false>(c, sms, s) : product<WK, T, false, 2, false>(c, sms, s);
}
template <int WK, bool FEW>
static cudaError_t down(const MoeCall& c, int sms, cudaStream_t s) {
  return c.n_tokens <= 8 ? product<WK, float, FEW, 1, true>(c, sms, s) : product<WK, float, FEW, 2, true>(c, sms, s);
}
template <typename T, int KE>
static cudaError_t router(const MoeCall& c, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = allow(k_moe_router<T, KE>, done, (EFFORT_MAX_IN_DIM + 8) * 4);
  if (e != cudaSuccess) return e;
  return start(k_moe_router<T, KE>, dim3((unsigned)c.n_tokens), kRouterThreads, (size_t)c.rpitch * 4, s, c);
}
template <int WK>
static cudaError_t all(const MoeCall& c, int sms, cudaStream_t s) {
  constexpr int KE = WK == kWE4M3 ? 128 : 64;
  cudaError_t e = c.xdt == kF32 ? router<float, KE>(c, s) : c.xdt == kF16 ? router<__half, KE>(c, s) : router<__nv_bfloat16, KE>(c, s);
  if (e == cudaSuccess)
    e = c.xdt == kF32 ? up<WK, float>(c, sms, s) : c.xdt == kF16 ? up<WK, __half>(c, sms, s) : up<WK, __nv_bfloat16>(c, sms, s);
  if (e == cudaSuccess) e = c.odt == kBF16 ? down<WK, true>(c, sms, s) : down<WK, false>(c, sms, s);
  if (e == cudaSuccess) e = start(k_moe_sum, dim3((unsigned)cdiv(c.I, 256), (unsigned)c.n_tokens), 256, 0, s, c);
  return e;
}

cudaError_t launch_moe(const MoeCall& c, int sms, cudaStream_t s) {
  return c.wk == kWE4M3 ? all<kWE4M3>(c, sms, s) : c.wk == kWF16 ? all<kWF16>(c, sms, s) : all<kWBF16>(c, sms, s);
}

size_t moe_scratch(MoeCall* c, char* base, int n_tokens, int top_k, int xdt_size, int n_experts, int I, int F, int wk,
                   int nkb13, int nkb2, int sms) {
  const int ke = k_per_block(wk), pairs = n_tokens * top_k;
  const int xpitch = nkb13 * ke, hpitch = nkb2 * ke;
  // K shares of the second product: the fewest that leave the SMs under 4% of
  // their time without a tile (by the experts that can be met), no share
  // shorter than one K block a warp
  const long long tiles = (long long)cdiv(I, 16) * (n_experts < pairs ? n_experts : pairs);
  const int most = nkb2 / 16 < 1 ? 1 : nkb2 / 16 > 16 ? 16 : nkb2 / 16;
  int shares = 1;
  double best = 0.0;
  for (int k = 1; k <= most; ++k) {
    const long long u = tiles * k;
    const double used = (double)u / (double)((u + sms - 1) / sms * sms);
    if (used > best + 1e-9) {
      best = used;
      shares = k;
    }
    if (best >= 0.96) break;
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t x0 = take((size_t)n_tokens * xpitch * xdt_size);
  const size_t h0 = take((size_t)pairs * hpitch * 4);
  const size_t z0 = take((size_t)shares * pairs * I * 4);
  if (c) {
    c->xop = base + x0;
    c->h = (float*)(base + h0);
    c->z = (float*)(base + z0);
    c->xpitch = xpitch;
    c->hpitch = hpitch;
    c->shares = shares;
  }
  return at;
}

}  // namespace effort
