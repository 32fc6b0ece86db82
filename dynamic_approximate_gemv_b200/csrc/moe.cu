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
constexpr int kRouterThreads = 1024;

// How x of type T (0 fp32, 1 binary16, 2 bfloat16) enters products with weights
// of kind WK: exactly, or fp32 in 22 (24) bits.
template <int WK, int T>
struct XKind {
  static constexpr bool kBF = WK == kWBF16;  // the matrix instruction's type
  static constexpr bool kSame = T == (kBF ? kBF16 : kF16);
  static constexpr bool kScaled = !kBF && !kSame;
  static constexpr int kParts = kSame ? 1 : T == kF32 ? (kBF ? 3 : 2) : kBF ? 2 : 1;
};
// How the hidden activations enter the second product: with bfloat16 weights in
// 16 or (out fp32) 24 bits, else in 22, or in 11 for a bfloat16 out, whose 8 bits
// they do not disturb: 261 against 297 us at 16 tokens of 8 x 4096 x 14336, top 2,
// e4m3, 80 against 84 at one.  (Layers whose columns differ much take 22 there too:
// see all().)
template <int WK, int ODT>
struct HKind {
  static constexpr bool kBF = WK == kWBF16, kScaled = !kBF;
  static constexpr int kParts = kBF ? (ODT == kF32 ? 3 : 2) : (ODT == kBF16 ? 1 : 2);
};

// One block per token: x in parts and its norm, the logits by warps, the top-k
// by one warp.
template <int WK, int T>
__global__ void __launch_bounds__(kRouterThreads) k_moe_router(const MoeCall c) {
  using X = XKind<WK, T>;
  constexpr int KE = WK == kWE4M3 ? 128 : 64, BLK = act_block<KE, X::kParts, X::kScaled>();
  extern __shared__ float xs[];  // the token, fp32, padded with zeros to whole K blocks
  __shared__ float logit[EFFORT_MAX_EXPERTS], wred[2][kRouterThreads / 32];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = warp_index(), E = c.n_experts, nkb = c.w13.nkb;
  constexpr int W = kRouterThreads / 32;
  grid_dep_launch();
  grid_dep_wait();
  float big = 0.0f;
  for (int k = threadIdx.x; k < nkb * KE; k += kRouterThreads) {
    const float v = k < c.I ? load_dt(c.x, T, t * c.xstride + k) : 0.0f;
    xs[k] = v;
    big = fmaxf(big, fabsf(v));
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, m));
  if (lane == 0) wred[0][warp] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) big = fmaxf(big, wred[0][w]);
  // the norm, of quotients by the largest value (or 1e-30), so that no square leaves the range
  const float unit = fmaxf(big, 1e-30f), inv = big < INFINITY ? __fdiv_rn(1.0f, unit) : 1.0f;
  float sq = 0.0f;
  char* to = c.xop + (size_t)t * c.xpitch;
  for (int kb = warp; kb < nkb; kb += W) {
    float up = 1.0f, down = 1.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < KE / 32; ++i) {
      const float v = xs[kb * KE + 32 * i + lane];
      m = fmaxf(m, fabsf(v));
      sq += v * inv * (v * inv);
    }
    if constexpr (X::kScaled) {
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
      pow2_scale(m, &up, &down);
      if (lane == 0) *reinterpret_cast<float*>(to + (size_t)kb * BLK + KE * 2 * X::kParts) = down;
    }
#pragma unroll
    for (int i = 0; i < KE / 32; ++i) {
      const int k = 32 * i + lane;
      store_parts<X::kBF, X::kParts>(reinterpret_cast<uint16_t*>(to + (size_t)kb * BLK) + frag_pos<KE>(k), KE,
                                     xs[kb * KE + k] * up);
    }
  }
#pragma unroll
  for (int m = 16; m; m >>= 1) sq += __shfl_xor_sync(~0u, sq, m);
  if (lane == 0) wred[1][warp] = sq;
  __syncthreads();
  if (threadIdx.x == 0) {
    float q = 0.0f;
    for (int w = 0; w < W; ++w) q += wred[1][w];
    c.xnorm[t] = big < INFINITY ? (double)unit * sqrt((double)q) : (double)big;
  }
  if (c.gate_mode == EFFORT_GATE_GIVEN) return;
  // a row of the router by one warp, or by several where there are few (their
  // sums are added in order); eight loads of a lane on their way at a time
  const int share = E >= W ? 1 : W / E, n16 = c.rpitch / (c.rdt == kF32 ? 4 : 8);  // 16-byte pieces
  __syncthreads();
  for (int task = warp; task < E * share; task += W) {
    const int e = task / share, p0 = n16 * (task % share) / share, p1 = n16 * (task % share + 1) / share;
    const uint4* r = reinterpret_cast<const uint4*>(c.router) + (size_t)e * n16;
    float s = 0.0f;
    for (int k0 = p0; k0 < p1; k0 += 256) {
      uint4 a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 32 * i + lane;
        a[i] = k < p1 ? __ldg(r + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 32 * i + lane;
        if (k >= p1) break;
        if (c.rdt == kF32) {
          const float4 b = reinterpret_cast<const float4*>(xs)[k];
          s += __uint_as_float(a[i].x) * b.x + __uint_as_float(a[i].y) * b.y + __uint_as_float(a[i].z) * b.z +
               __uint_as_float(a[i].w) * b.w;
        } else {
          const float4 b0 = reinterpret_cast<const float4*>(xs)[2 * k], b1 = reinterpret_cast<const float4*>(xs)[2 * k + 1];
          float2 f[4];
          if (c.rdt == kBF16) f[0] = unpack2<true>(a[i].x), f[1] = unpack2<true>(a[i].y), f[2] = unpack2<true>(a[i].z), f[3] = unpack2<true>(a[i].w);
          else f[0] = unpack2<false>(a[i].x), f[1] = unpack2<false>(a[i].y), f[2] = unpack2<false>(a[i].z), f[3] = unpack2<false>(a[i].w);
          s += f[0].x * b0.x + f[0].y * b0.y + f[1].x * b0.z + f[1].y * b0.w;
          s += f[2].x * b1.x + f[2].y * b1.y + f[3].x * b1.z + f[3].y * b1.w;
        }
      }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(~0u, s, m);
    if (lane == 0) logit[task] = s;
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
    l[i] = -INFINITY;
    if (e < E) {
      l[i] = logit[e * share];
      for (int p = 1; p < share; ++p) l[i] += logit[e * share + p];
    }
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

// place, id: kMaxPairs each; cnt: EFFORT_MAX_EXPERTS
__device__ void make_plan(Plan* p, const int* ids, int pairs, int E, int cols, uint16_t* place, int16_t* id, int* cnt,
                          int warp, int lane, int threads) {
  for (int e = threadIdx.x; e < E; e += threads) cnt[e] = 0;
  for (int i = threadIdx.x; i < pairs; i += threads) {
    const int v = ids[i];
    id[i] = (int16_t)(v >= 0 && v < E ? v : -1);
  }
  __syncthreads();
  if (warp == 0) {
    // a pair's place among those of its expert
    for (int b = 0; b < pairs; b += 32) {
      const int e = b + lane < pairs ? id[b + lane] : -1;
      const unsigned same = __match_any_sync(~0u, e >= 0 ? e : -1 - lane);
      const int before = __popc(same & ((1u << lane) - 1)), base = e >= 0 ? cnt[e] : 0;
      __syncwarp();
      if (e >= 0) {
        place[b + lane] = (uint16_t)(base + before);
        if (before == 0) cnt[e] = base + __popc(same);
      }
      __syncwarp();
    }
    // starts of the lists and of the chunks
    int list0 = 0, chunk0 = 0;
    for (int b = 0; b < E; b += 32) {
      const int e = b + lane, k = e < E ? cnt[e] : 0, m = (k + cols - 1) / cols;
      int n1 = k, m1 = m;  // sums up to and with this lane
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(~0u, n1, d), y = __shfl_up_sync(~0u, m1, d);
        if (lane >= d) n1 += x, m1 += y;
      }
      const int n0 = list0 + n1 - k, m0 = chunk0 + m1 - m;
      for (int i = 0; i < m; ++i)
        p->chunk[m0 + i] = (uint32_t)(n0 + i * cols) << 13 | (uint32_t)min(cols, k - i * cols) << 8 | (uint32_t)e;
      if (e < E) cnt[e] = n0;
      list0 += __shfl_sync(~0u, n1, 31);
      chunk0 += __shfl_sync(~0u, m1, 31);
    }
    if (lane == 0) p->chunks = chunk0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += threads)
    if (id[i] >= 0) p->list[cnt[id[i]] + place[i]] = (uint16_t)i;
  __syncthreads();
}

// ---------------------------------------------------------------- products
constexpr int kPlanBytes = (int)(sizeof(Plan) + 15) / 16 * 16, kMoeExtra = kPlanBytes + EFFORT_MAX_TOKENS * 8;
template <int WK, int PARTS, int ROWS>
using MoeShape = StreamShape<ROWS, (WK == kWE4M3 ? 128 : 64) * 2 * PARTS, 64, kMoeExtra>;

// The power of two that brings the hidden activations of one token and K block
// into binary16's range before they are known: |silu(a) b| <= |a| |b|, each at
// most the norm of x times the largest column norm of the block.  The bound is
// held in 64 bits: one factor may lie far from 1 where the product does not.  It
// comes to lie in [2^14, 2^15), half of binary16's largest value or less, which
// leaves room for the roundings; typical values lie 2^9 to 2^12 below it, and
// lower by as much as some column of the block, or some input, stands out.
__device__ __forceinline__ void hidden_scale(double xnorm, double2 n, float* up, float* down) {
  const double b = xnorm * n.x * (xnorm * n.y);
  // b < 2^k, at least 2^-96 as in pow2_scale; the values themselves are fp32 (inf and
  // NaN end up somewhere)
  const int k = max(-96, min((__double2hiint(b) >> 20 & 0x7ff) - 1022, 128));
  *up = __uint_as_float((uint32_t)(127 + 15 - k) << 23);
  *down = __uint_as_float((uint32_t)(127 - 15 + k) << 23);
}

// PARTS, SCALED: of the activations read; HPARTS, HSCALED (first product): of
// the hidden activations written.  ROWS: rows of a chunk.  DOWN: the second product.
template <int WK, int PARTS, bool SCALED, int HPARTS, bool HSCALED, int ROWS, bool DOWN>
__global__ void __launch_bounds__(MoeShape<WK, PARTS, ROWS>::kThreads, 1) k_moe_product(const MoeCall c) {
  using S = MoeShape<WK, PARTS, ROWS>;
  constexpr int NT = S::NT, MT = S::kMT, W = S::kWarps, KE = WK == kWE4M3 ? 128 : 64, KS = KE / 16;
  constexpr int BLK = act_block<KE, PARTS, SCALED>(), HBLK = act_block<KE, HPARTS, HSCALED>();
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  float* red = reinterpret_cast<float*>(smem + S::kRedAt);
  Plan* plan = reinterpret_cast<Plan*>(smem + S::kExtraAt);
  double* xnorm = reinterpret_cast<double*>(smem + S::kExtraAt + kPlanBytes);
  const int lane = threadIdx.x & 31, warp = warp_index(), g = lane >> 2, q = lane & 3;
  const TileMat w = DOWN ? c.w2 : c.w13;
  const int nkb = w.nkb, nkb4 = align4(nkb), pairs = c.n_tokens * c.top_k;
  const int tiles = DOWN ? cdiv(c.I, 16) : cdiv(c.F, 8), shares = DOWN ? c.shares : 1;

  grid_dep_launch();
  grid_dep_wait();
  if (!DOWN && HSCALED)
    for (int i = threadIdx.x; i < c.n_tokens; i += S::kThreads) xnorm[i] = c.xnorm[i];
  uint8_t* temp = smem + S::kRingAt;  // the ring is not in use yet
  make_plan(plan, c.ids, pairs, c.n_experts, ROWS, reinterpret_cast<uint16_t*>(temp),
            reinterpret_cast<int16_t*>(temp + 2 * kMaxPairs), reinterpret_cast<int*>(temp + 4 * kMaxPairs), warp, lane,
            S::kThreads);
  Ring<S> ring;
  ring.init(sbase, warp, lane);
  const int units = plan->chunks * shares * tiles;
  const int u0 = (int)((long long)units * blockIdx.x / gridDim.x), u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);

  // A group: up to MT tiles of one chunk (and K share), inside 64 stored rows.
  // kw warps share a group's K blocks; where those are few the block's warps
  // form several sets, which take the groups in turn, so that a warp has three
  // K blocks or more for each join.
  int kw = W;
  while (kw % 2 == 0 && nkb / shares < 3 * kw && (2 * W / kw) * MT <= u1 - u0) kw /= 2;
  const int sets = W / kw, set = warp / kw, wk = warp % kw;
  // The units' order: expert, K share, 64 stored rows, chunk of the expert, tile;
  // so an expert of several chunks finds its weights in L2 for all but the first.
  struct Cursor {
    int u, c0, m, share, b, ch, t, n;  // c0, m: the expert's first chunk and their number; b: 64 rows
  };
  const int chunks = plan->chunks;
  auto same = [&](int c, int d) { return ((plan->chunk[c] ^ plan->chunk[d]) & 255) == 0; };
  auto run = [&](int c0) {
    int m = 1;
    while (c0 + m < chunks && same(c0, c0 + m)) ++m;
    return m;
  };
  auto size = [&](Cursor& c) { c.n = min(min(MT, min(4 * c.b + 4, tiles) - c.t), u1 - c.u); };
  auto next = [&](Cursor& c) {
    c.u += c.n;
    c.t += c.n;
    if (c.t == min(4 * c.b + 4, tiles)) {
      if (++c.ch == c.m) {
        c.ch = 0;
        if (4 * ++c.b >= tiles) {
          c.b = 0;
          if (++c.share == shares) {
            c.share = 0;
            c.c0 += c.m;
            if (c.c0 < chunks) c.m = run(c.c0);
          }
        }
      }
      c.t = 4 * c.b;
    }
    size(c);
  };
  Cursor first = {u0, 0, 1, 0, 0, 0, 0, 0};
  if (u0 < u1) {
    int c0 = u0 / (shares * tiles);
    while (c0 > 0 && same(c0 - 1, c0)) --c0;
    const int m = run(c0), local = u0 - c0 * shares * tiles, share = local / (m * tiles), l = local - share * m * tiles;
    const int b = l / (4 * m), nb = min(4, tiles - 4 * b), r = l - 4 * m * b;
    first = {u0, c0, m, share, b, r / nb, 4 * b + r % nb, 0};
    size(first);
  }
  for (int i = 0; i < set && first.u < u1; ++i) next(first);
  struct Group {
    int expert, start, count, t, n, kb0, kb1, share;
  };
  auto group_at = [&](const Cursor& cu) {
    Group G;
    G.t = cu.t;
    G.n = cu.n;
    G.share = cu.share;
    const uint32_t ch = plan->chunk[cu.c0 + cu.ch];
    G.expert = ch & 255;
    G.count = ch >> 8 & 31;
    G.start = ch >> 13;
    G.kb0 = DOWN ? nkb * G.share / shares : 0;
    G.kb1 = DOWN ? nkb * (G.share + 1) / shares : nkb;
    return G;
  };
  auto step = [&](Cursor& cu) {
    for (int i = 0; i < sets && cu.u < u1; ++i) next(cu);
  };
  // what the warp asks for next
  Cursor pc = first;
  int pk = 0;
  Group P = {};
  auto seek = [&]() {  // the first group from pc on that has a K block for this warp
    while (pc.u < u1) {
      P = group_at(pc);
      pk = P.kb0 + wk;
      if (pk < P.kb1) return;
      step(pc);
    }
  };
  auto ask = [&]() {
    if (pc.u >= u1) return;
    const uint32_t buf = ring.next_buf(), bar = ring.next_bar();
    constexpr int kScales = WK == kWE4M3 ? (DOWN ? 1 : 2) : 0;
    if (lane == 0) {
      mbar_expect(bar, P.n * 2 * kCoreBytes + P.count * BLK + 16 * kScales + c.hook.lost(ring.put));
      bulk_load(buf, w.data + P.expert * w.stride + core_at(2 * P.t, pk, nkb), P.n * 2 * kCoreBytes, bar);
    }
    __syncwarp();
    if (lane >= 8 && lane - 8 < P.count) {
      const int p = plan->list[P.start + lane - 8];
      const char* row = DOWN ? c.h + (size_t)p * c.hpitch : c.xop + (size_t)(p / c.top_k) * c.xpitch;
      bulk_load(buf + S::kActAt + (lane - 8) * S::kRowPitch, row + (size_t)pk * BLK, BLK, bar);
    }
    if (kScales > 0 && lane >= 1 && lane <= kScales) {
      const float* s = DOWN ? c.s2 : lane == 1 ? c.s1 : c.s3;
      const int nsb = DOWN ? c.nsb2 : c.nsb13, blk = DOWN ? P.t / 8 : P.t / 16;
      bulk_load(buf + S::kScaleAt + 16 * (lane - 1), s + ((size_t)P.expert * nsb + blk) * nkb4 + (pk & ~3), 16, bar);
    }
    ++ring.put;
    pk += kw;
    if (pk >= P.kb1) {
      step(pc);
      seek();
    }
  };
  seek();
#pragma unroll 1
  for (int s = 0; s < S::kStages; ++s) ask();

  for (Cursor cu = first; cu.u < u1; step(cu)) {
    const Group G = group_at(cu);
    const int live = NT == 1 ? 1 : (G.count + 7) / 8;
    double2 bound = make_double2(0.0, 0.0);
    if (!DOWN && HSCALED) bound = __ldg(c.bound + (size_t)G.expert * c.w2.nkb + G.t * 8 / KE);
    float acc[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    for (int kb = G.kb0 + wk; kb < G.kb1; kb += kw) {
      const uint32_t at = ring.wait(smem, warp, c.hook, [&]() { pc.u = u1; });
      uint32_t b[PARTS][NT][KS][2];
      // the scales of column 2 q + e and the tile's rows g, g + 8: x's power of two times
      // the weights', as far as it is above 1, and before that what is below (so
      // that no product of two of the three leaves fp32's range where all three do not)
      constexpr bool kLess = SCALED && WK == kWE4M3;
      float sc[NT][2][2], less[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        act_load<PARTS, NT, KS>(at + S::kActAt + (8 * j + g) * S::kRowPitch, q, 8 * j + g < G.count, b, j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // of the columns this lane has sums of
          const int r = 8 * j + 2 * q + e;
          const float sx = SCALED && r < G.count ? lds_float(at + S::kActAt + r * S::kRowPitch + KE * 2 * PARTS) : 1.0f;
          less[j][e] = kLess ? fminf(sx, 1.0f) : 1.0f;
          sc[j][e][0] = sc[j][e][1] = kLess ? fmaxf(sx, 1.0f) : sx;
        }
      }
      if constexpr (WK == kWE4M3) {
        const float s0 = lds_float(at + S::kScaleAt + 4 * (kb & 3));
        const float s1 = DOWN ? s0 : lds_float(at + S::kScaleAt + 16 + 4 * (kb & 3));
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[j][e][0] *= s0;
            sc[j][e][1] *= s1;
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= G.n) break;
        // the sum of one K block apart, to be scaled, and because the matrix
        // instruction truncates: over many K blocks that adds up
        float d[NT][4] = {};
        mma_tile<WK, NT, PARTS, KS>(at + m * 2 * kCoreBytes, g, q, b, live, d);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[m][j][e] = fmaf(d[j][e] * less[j][e & 1], sc[j][e & 1][e >> 1], acc[m][j][e]);
      }
      __syncwarp();  // every lane has read the stage
      ask();
    }
    // join the set's sums
    set_sync(set, kw);
    float* mine = red + warp * S::kRed;
    const float poison = ring.fine ? 0.0f : __int_as_float(0x7fffffff);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(8 * j + 2 * q + (e & 1)) * S::kPitch + 16 * m + g + 8 * (e >> 1)] = acc[m][j][e] + poison;
    set_sync(set, kw);
    constexpr int kWide = DOWN ? MT * 16 : MT * 8;  // outputs of a column
    for (int i = wk * 32 + lane; i < G.count * kWide; i += kw * 32) {
      const int col = i / kWide, o = i % kWide;
      const float* r = red + set * kw * S::kRed + col * S::kPitch + (DOWN ? o : o / 8 * 16 + o % 8);
      float a = 0.0f, b = 0.0f;
      if (kw == W) {
#pragma unroll
        for (int v = 0; v < W; ++v) {
          a += r[v * S::kRed];
          if (!DOWN) b += r[v * S::kRed + 8];
        }
      } else {
        for (int v = 0; v < kw; ++v) {
          a += r[v * S::kRed];
          if (!DOWN) b += r[v * S::kRed + 8];
        }
      }
      const int p = plan->list[G.start + col];
      if constexpr (DOWN) {
        const int row = G.t * 16 + o;
        if (o < G.n * 16 && row < c.I) c.z[((size_t)G.share * pairs + p) * c.I + row] = a;
      } else if (o < G.n * 8) {
        // behind the last hidden unit the weights are zero and so is the sum;
        // the last K block is written to its end by its last tiles' threads
        const int j = G.t * 8 + o, kb = j / KE;
        char* blk = c.h + (size_t)p * c.hpitch + (size_t)kb * HBLK;
        float up = 1.0f, down = 1.0f;
        if (HSCALED) {
          hidden_scale(xnorm[p / c.top_k], bound, &up, &down);
          if (j % KE == 0) *reinterpret_cast<float*>(blk + KE * 2 * HPARTS) = down;
        }
        const float v = j < c.F ? __fdiv_rn(a, 1.0f + expf(-a)) * b : 0.0f;
        store_parts<WK == kWBF16, HPARTS>(reinterpret_cast<uint16_t*>(blk) + frag_pos<KE>(j % KE), KE, v * up);
        if (G.t + G.n == tiles && o / 8 == G.n - 1)  // the K block's rest
          for (int k = j + 8; k < (kb + 1) * KE; k += 8)
            store_parts<WK == kWBF16, HPARTS>(reinterpret_cast<uint16_t*>(blk) + frag_pos<KE>(k % KE), KE, 0.0f);
      }
    }
  }
  ring.drain(smem, warp, lane, c.hook);
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

// ---------------------------------------------------------------- preparation
__device__ __forceinline__ float weight_value(const void* w, int wk, size_t i) {
  if (wk == kWE4M3) return e4m3_to_float(static_cast<const uint8_t*>(w)[i]);
  return wk == kWF16 ? __half2float(static_cast<const __half*>(w)[i]) : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}
// The largest column norms of w1 (and w3: blockIdx.z = 1) over each K block of
// hidden units, in 64 bits, since squares of values and scales that fp32 holds may
// leave its range.  One block of 256 threads per (K block, expert, matrix).  Bit 1
// of status is set where norms of one K block (but zero) differ by more than kSpread.
constexpr double kSpread = 32.0;
__global__ void __launch_bounds__(256) k_moe_bounds(const void* w1, const void* w3, const float* s1, const float* s3, int wk,
                                                    int I, int F, double2* bound, unsigned* status) {
  const int KE = k_per_block(wk), kb = blockIdx.x, e = blockIdx.y, parts = 256 / KE;
  const void* w = blockIdx.z ? w3 : w1;
  const float* s = blockIdx.z ? s3 : s1;
  const int j = kb * KE + threadIdx.x % KE, part = threadIdx.x / KE;
  __shared__ double sums[256];
  double q = 0.0;
  if (j < F)
    for (int i = part; i < I; i += parts) {
      double v = weight_value(w, wk, ((size_t)e * I + i) * F + j);
      if (wk == kWE4M3) v *= s[((size_t)e * cdiv(I, kBlk) + i / kBlk) * cdiv(F, kBlk) + j / kBlk];
      q += v * v;
    }
  sums[threadIdx.x] = q;
  __syncthreads();
  if (threadIdx.x == 0) {
    double m = 0.0, low = INFINITY;
    for (int k = 0; k < KE; ++k) {
      double t = 0.0;
      for (int p = 0; p < parts; ++p) t += sums[p * KE + k];
      m = fmax(m, t);
      if (t > 0.0) low = fmin(low, t);
    }
    if (m > kSpread * kSpread * low) atomicOr(status, 2u);
    double* b = reinterpret_cast<double*>(bound + (size_t)e * gridDim.x + kb);
    b[blockIdx.z] = sqrt(m);
  }
}
cudaError_t launch_moe_bounds(const void* w1, const void* w3, const float* s1, const float* s3, int wk, int E, int I, int F,
                              double2* bound, unsigned* status, cudaStream_t s) {
  k_moe_bounds<<<dim3((unsigned)cdiv(F, k_per_block(wk)), (unsigned)E, 2), 256, 0, s>>>(w1, w3, s1, s3, wk, I, F, bound,
                                                                                           status);
  return cudaGetLastError();
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

template <int WK, int PARTS, bool SCALED, int HPARTS, bool HSCALED, int ROWS, bool DOWN>
static cudaError_t product(const MoeCall& c, int sms, cudaStream_t s) {
  using S = MoeShape<WK, PARTS, ROWS>;
  static_assert(S::kWarps * S::kStages * S::kStage >= 4 * kMaxPairs + 4 * EFFORT_MAX_EXPERTS, "the plan's working space");
  static std::atomic<bool> done[kMaxDevices];
  const auto kernel = k_moe_product<WK, PARTS, SCALED, HPARTS, HSCALED, ROWS, DOWN>;
  cudaError_t e = allow(kernel, done, S::kSmem);
  if (e != cudaSuccess) return e;
  return start(kernel, dim3((unsigned)sms), S::kThreads, S::kSmem, s, c);
}
// Rows of a chunk: they are read beside every K block and have their place in
// its stage, so fewer leave room for more warps; the weights of a longer list
// are read again.  With lists of up to 4 pairs on average 8 rows are better
// (16 tokens, top 2 of 8 experts of 4096 x 14336: 257 against 446 us in e4m3,
// 452 against 517 us in binary16; one list in 140 is longer than 8).
template <int WK, int PARTS, bool SCALED, int HPARTS, bool HSCALED, bool DOWN>
static cudaError_t by_rows(const MoeCall& c, int sms, cudaStream_t s) {
  if (c.n_tokens == 1) return product<WK, PARTS, SCALED, HPARTS, HSCALED, 1, DOWN>(c, sms, s);
  if (c.n_tokens <= 8 || c.n_tokens * c.top_k <= 4 * c.n_experts) return product<WK, PARTS, SCALED, HPARTS, HSCALED, 8, DOWN>(c, sms, s);
  return product<WK, PARTS, SCALED, HPARTS, HSCALED, 16, DOWN>(c, sms, s);
}
template <int WK, int T, int ODT>
static cudaError_t all(const MoeCall& c, int sms, cudaStream_t s) {
  using X = XKind<WK, T>;
  using H = HKind<WK, ODT>;
  // 11 bits reach 2^28 below the bound of a K block's hidden activations, where
  // typical ones lie 2^9 to 2^12 below their own columns'
  if constexpr (!H::kBF && ODT == kBF16) {
    if (c.spread) return all<WK, T, kF16>(c, sms, s);
  }
  static std::atomic<bool> done[kMaxDevices];
  const size_t smem = (size_t)c.w13.nkb * k_per_block(WK) * 4;
  cudaError_t e = allow(k_moe_router<WK, T>, done, (EFFORT_MAX_IN_DIM + 128) * 4);
  if (e == cudaSuccess) e = start(k_moe_router<WK, T>, dim3((unsigned)c.n_tokens), kRouterThreads, smem, s, c);
  if (e == cudaSuccess) e = by_rows<WK, X::kParts, X::kScaled, H::kParts, H::kScaled, false>(c, sms, s);
  if (e == cudaSuccess) e = by_rows<WK, H::kParts, H::kScaled, 1, false, true>(c, sms, s);
  if (e == cudaSuccess) e = start(k_moe_sum, dim3((unsigned)cdiv(c.I, 256), (unsigned)c.n_tokens), 256, 0, s, c);
  return e;
}
template <int WK, int T>
static cudaError_t by_out(const MoeCall& c, int sms, cudaStream_t s) {
  return c.odt == kF32 ? all<WK, T, kF32>(c, sms, s) : c.odt == kF16 ? all<WK, T, kF16>(c, sms, s) : all<WK, T, kBF16>(c, sms, s);
}
template <int WK>
static cudaError_t by_x(const MoeCall& c, int sms, cudaStream_t s) {
  return c.xdt == kF32 ? by_out<WK, kF32>(c, sms, s) : c.xdt == kF16 ? by_out<WK, kF16>(c, sms, s) : by_out<WK, kBF16>(c, sms, s);
}

cudaError_t launch_moe(const MoeCall& c, int sms, cudaStream_t s) {
  return c.wk == kWE4M3 ? by_x<kWE4M3>(c, sms, s) : c.wk == kWF16 ? by_x<kWF16>(c, sms, s) : by_x<kWBF16>(c, sms, s);
}

size_t moe_scratch(MoeCall* c, char* base, int n_tokens, int top_k, int n_experts, int I, int F, int wk, int nkb13,
                   int nkb2, int sms) {
  const int ke = k_per_block(wk), pairs = n_tokens * top_k;
  // K blocks in their longest form
  const int blk = wk == kWBF16 ? ke * 2 * 3 : ke * 2 * 2 + 16;
  const int xpitch = nkb13 * blk, hpitch = nkb2 * blk;
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
  const size_t x0 = take((size_t)n_tokens * xpitch);
  const size_t n0 = take((size_t)n_tokens * 8);
  const size_t h0 = take((size_t)pairs * hpitch);
  const size_t z0 = take((size_t)shares * pairs * I * 4);
  if (c) {
    c->xop = base + x0;
    c->xnorm = (double*)(base + n0);
    c->h = base + h0;
    c->z = (float*)(base + z0);
    c->xpitch = xpitch;
    c->hpitch = hpitch;
    c->shares = shares;
    c->hook = wait_hook();
  }
  return at;
}

}  // namespace effort
