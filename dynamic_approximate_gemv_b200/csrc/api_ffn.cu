// Host side of the feed-forward operators: argument checks, storage of the
// weights, and the launches.
#include <math.h>

#include <new>

#include "../../include/effort.h"
#include "ffn_common.cuh"
#include "host.cuh"
#include "moe.cuh"

namespace effort {
cudaError_t launch_block_norm(const effort_block_norm_t& a, int sms, cudaStream_t s);
cudaError_t launch_tile_weights(int wk, const void* w, int mats, int K, int N, uint8_t* out, int cores, int nkb,
                                size_t stride, int pair, unsigned* status, cudaStream_t s);
cudaError_t launch_check_finite(const float* p, size_t n, unsigned* status, cudaStream_t s);
cudaError_t launch_turn_scales(const float* s, int mats, int nkb, int nsb, float* out, cudaStream_t st);
cudaError_t launch_fp8_matmul(const TileMat& w, const float* ws, int I, int O, const uint8_t* x, int64_t xstride,
                              const float* xs, int64_t xsstride, int64_t rows, int odt, void* out, int64_t ostride,
                              cudaStream_t s);
cudaError_t launch_moe(const MoeCall& c, int sms, cudaStream_t s);
cudaError_t launch_moe_bounds(const void* w1, const void* w3, const float* s1, const float* s3, int wk, int E, int I, int F,
                              double2* bound, unsigned* status, cudaStream_t s);
}  // namespace effort

using namespace effort;

struct effort_fp8_s {
  int dev = 0;
  int64_t I = 0, O = 0;
  DevBuf buf;  // cores, then the scales
  TileMat w = {};
  const float* ws = nullptr;
};

struct effort_moe_s {
  int dev = 0;
  int sms = 0, E = 0, wk = 0, rdt = 0, rpitch = 0;
  int64_t I = 0, F = 0;
  DevBuf buf;  // cores of w1/w3, cores of w2, scales, router
  TileMat w13 = {}, w2 = {};
  const float *s1 = nullptr, *s3 = nullptr, *s2 = nullptr;
  const double2* bound = nullptr;
  bool spread = false;
  const void* router = nullptr;
};

namespace {

bool dtype_ok(int t) { return t == EFFORT_F32 || t == EFFORT_F16 || t == EFFORT_BF16; }
size_t dtype_size(int t) { return t == EFFORT_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool kind_ok(int k) { return k == EFFORT_NORM_NONE || k == EFFORT_NORM_RMS || k == EFFORT_NORM_LAYER; }

// An array of a call: rows of `width` bytes, `stride` bytes apart (at least width).
struct Span {
  const void* p;
  int64_t rows, stride, width;
  uintptr_t lo, hi;  // all of it; empty where p is null
  Span(const void* p_, int64_t rows_, int64_t stride_, int64_t width_) : p(p_), rows(rows_), stride(stride_), width(width_) {
    lo = hi = (uintptr_t)p;
    uint64_t n;
    if (p && (__builtin_mul_overflow((uint64_t)(rows - 1), (uint64_t)stride, &n) || __builtin_add_overflow(n, (uint64_t)width, &n) ||
              __builtin_add_overflow(lo, n, &hi)))
      hi = UINTPTR_MAX;
  }
};

// Whether two arrays whose ranges overlap have a byte in common.
bool rows_meet(const Span& a, const Span& b) {
  if (a.rows == 1 && b.rows == 1) return true;
  using Wide = __int128;
  const Wide d = (Wide)b.lo - (Wide)a.lo, sa = a.rows > 1 ? a.stride : b.stride, sb = b.rows > 1 ? b.stride : a.stride;
  if (sa == sb) {
    // row i of a, i + k of b: k's least value with d + k s > -b.width, and in b
    const Wide num = -(Wide)b.width - d;
    Wide k = num / sa - (num % sa < 0 ? 1 : 0) + 1;
    if (k < 1 - a.rows) k = 1 - a.rows;
    return k < b.rows && d + k * sa < a.width;
  }
  for (int64_t i = 0, j = 0; i < a.rows && j < b.rows;) {
    const Wide at = d + j * sb - i * sa;  // b's row seen from a's
    if (at >= a.width) ++i;
    else if (at <= -(Wide)b.width) ++j;
    else return true;
  }
  return false;
}
inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi && rows_meet(a, b); }

effort_status_t device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return EFFORT_ERR_CUDA;
  }
  return EFFORT_OK;
}

size_t call_scratch(effort_moe_t h, MoeCall* c, char* base, int n_tokens, int top_k) {
  return moe_scratch(c, base, n_tokens, top_k, h->E, (int)h->I, (int)h->F, h->wk, h->w13.nkb, h->w2.nkb, h->sms);
}

effort_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return EFFORT_OK;
  cudaGetLastError();
  return EFFORT_ERR_CUDA;
}

}  // namespace

extern "C" {

effort_status_t effort_block_norm(const effort_block_norm_t* args, void* stream) {
  if (!args) return EFFORT_ERR_ARG;
  const effort_block_norm_t& a = *args;
  if (a.rows < 0 || a.dim < 1 || !a.x) return EFFORT_ERR_ARG;
  if (!dtype_ok(a.dtype) || !dtype_ok(a.weight_dtype) || (a.h_out && !dtype_ok(a.h_dtype))) return EFFORT_ERR_ARG;
  if (!kind_ok(a.post_kind) || !kind_ok(a.pre_kind)) return EFFORT_ERR_ARG;
  if (!a.x_out && !a.h_out && !a.q_out) return EFFORT_ERR_ARG;
  if ((a.q_out != nullptr) != (a.q_scales != nullptr)) return EFFORT_ERR_ARG;
  // what works on y is not given without it
  if (!a.y && (a.gate || a.post_kind != EFFORT_NORM_NONE)) return EFFORT_ERR_ARG;
  if (!(a.eps >= 0.0f) || !isfinite(a.eps) || !isfinite(a.weight_offset) || !isfinite(a.residual_scale) ||
      !isfinite(a.branch_scale))
    return EFFORT_ERR_ARG;
  const size_t sz = dtype_size(a.dtype), wsz = dtype_size(a.weight_dtype);
  if (!aligned(a.x, sz) || !aligned(a.y, sz) || !aligned(a.gate, sz) || !aligned(a.x_out, sz)) return EFFORT_ERR_ARG;
  if (!aligned(a.post_weight, wsz) || !aligned(a.post_bias, wsz) || !aligned(a.pre_weight, wsz) ||
      !aligned(a.pre_bias, wsz))
    return EFFORT_ERR_ARG;
  if (a.h_out && !aligned(a.h_out, dtype_size(a.h_dtype))) return EFFORT_ERR_ARG;
  if (!aligned(a.q_scales, 4)) return EFFORT_ERR_ARG;
  if (a.x_stride < a.dim || (a.y && a.y_stride < a.dim) || (a.x_out && a.x_out_stride < a.dim) ||
      (a.h_out && a.h_stride < a.dim) || (a.q_out && a.q_stride < a.dim) ||
      (a.gate && a.gate_stride != 0 && a.gate_stride < a.dim) ||
      (a.q_out && a.q_scales_stride < (a.dim + kBlk - 1) / kBlk))
    return EFFORT_ERR_ARG;
  if (a.rows > EFFORT_MAX_ROWS || a.dim > EFFORT_MAX_IN_DIM) return EFFORT_ERR_UNSUPPORTED;
  if (a.rows == 0) return EFFORT_OK;
  const size_t hsz = a.h_out ? dtype_size(a.h_dtype) : 0;
  auto rows = [&](const void* p, int64_t stride, size_t size) {
    return Span{p, a.rows, stride * (int64_t)size, a.dim * (int64_t)size};
  };
  auto vec = [&](const void* p) { return Span{p, 1, 0, a.dim * (int64_t)wsz}; };
  const Span in[] = {rows(a.x, a.x_stride, sz), rows(a.y, a.y_stride, sz),
                     {a.gate, a.gate_stride ? a.rows : 1, a.gate_stride * (int64_t)sz, a.dim * (int64_t)sz},
                     vec(a.post_weight), vec(a.post_bias), vec(a.pre_weight), vec(a.pre_bias)};
  const Span out[] = {rows(a.x_out, a.x_out_stride, sz), rows(a.h_out, a.h_stride, hsz), rows(a.q_out, a.q_stride, 1),
                      {a.q_scales, a.rows, a.q_scales_stride * 4, (a.dim + kBlk - 1) / kBlk * 4}};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 7; ++i) {
      // x_out and h_out in the place of x or y: an element is read before it is written
      const bool same = o < 2 && i < 2 && in[i].p == out[o].p && in[i].width == out[o].width &&
                        (a.rows == 1 || in[i].stride == out[o].stride);
      if (!same && meet(in[i], out[o])) return EFFORT_ERR_ARG;
    }
    for (int i = 0; i < o; ++i)
      if (meet(out[i], out[o])) return EFFORT_ERR_ARG;
  }
  int sms = 0;
  effort_status_t st = device_sms(&sms);
  if (st != EFFORT_OK) return st;
  return launched(launch_block_norm(a, sms, (cudaStream_t)stream));
}

effort_status_t effort_fp8_prepare(const void* q, const float* scales, int64_t in_dim, int64_t out_dim, void* stream,
                                   effort_fp8_t* out_matrix) {
  if (!out_matrix) return EFFORT_ERR_ARG;
  *out_matrix = nullptr;
  if (!q || !scales || !aligned(scales, 4) || in_dim < 1 || out_dim < 1) return EFFORT_ERR_ARG;
  if (in_dim > EFFORT_MAX_FP8_DIM || out_dim > EFFORT_MAX_FP8_DIM || in_dim * out_dim >= (1ll << 36))
    return EFFORT_ERR_UNSUPPORTED;
  const int nkb = cdiv(in_dim, kBlk), nsb = cdiv(out_dim, kBlk), cores = nsb * 16;
  const size_t wbytes = (size_t)cores * nkb * kCoreBytes, sbytes = align_up((size_t)align4(nkb) * nsb * 4, 256);
  if (!within_cap(wbytes + sbytes + 256)) return EFFORT_ERR_NOMEM;
  effort_fp8_s* m = new (std::nothrow) effort_fp8_s();
  if (!m) return EFFORT_ERR_NOMEM;
  auto fail = [&](effort_status_t s) {
    cudaGetLastError();
    m->buf.release();
    delete m;
    return s;
  };
  if (cudaGetDevice(&m->dev) != cudaSuccess) return fail(EFFORT_ERR_CUDA);
  effort_status_t st = m->buf.alloc(wbytes + sbytes + 256);
  if (st != EFFORT_OK) return fail(st);
  m->I = in_dim;
  m->O = out_dim;
  m->w = {(const uint8_t*)m->buf.p, cores, nkb, wbytes};
  m->ws = (const float*)((char*)m->buf.p + wbytes);
  unsigned* status = (unsigned*)((char*)m->buf.p + wbytes + sbytes);
  cudaStream_t s = (cudaStream_t)stream;
  unsigned bad = 0;
  cudaError_t e = cudaMemsetAsync(status, 0, 4, s);
  if (e == cudaSuccess)
    e = launch_tile_weights(kWE4M3, q, 1, (int)in_dim, (int)out_dim, (uint8_t*)m->buf.p, cores, nkb, wbytes, 0, status, s);
  if (e == cudaSuccess) e = launch_check_finite(scales, (size_t)nkb * nsb, status, s);
  if (e == cudaSuccess) e = launch_turn_scales(scales, 1, nkb, nsb, (float*)m->ws, s);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&bad, status, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(EFFORT_ERR_CUDA);
  if (bad) return fail(EFFORT_ERR_NONFINITE);
  *out_matrix = m;
  return EFFORT_OK;
}

effort_status_t effort_fp8_matmul(effort_fp8_t m, const void* x, int64_t x_stride, const float* x_scales,
                                  int64_t x_scales_stride, int64_t rows, effort_dtype_t out_dtype, void* out,
                                  int64_t out_stride, void* stream) {
  if (!m || rows < 0 || !dtype_ok(out_dtype)) return EFFORT_ERR_ARG;
  if (rows > 0 && (!x || !x_scales || !out)) return EFFORT_ERR_ARG;
  if (!aligned(x, 16) || x_stride % 16 != 0 || x_stride < m->I || !aligned(x_scales, 4) || x_scales_stride < m->w.nkb)
    return EFFORT_ERR_ARG;
  if (!aligned(out, dtype_size(out_dtype)) || out_stride < m->O) return EFFORT_ERR_ARG;
  if (rows > EFFORT_MAX_ROWS) return EFFORT_ERR_UNSUPPORTED;
  if (rows == 0) return EFFORT_OK;
  const int64_t osz = (int64_t)dtype_size(out_dtype);
  const Span o = {out, rows, out_stride * osz, m->O * osz};
  if (meet(o, {x, rows, x_stride, m->I}) || meet(o, {x_scales, rows, x_scales_stride * 4, m->w.nkb * 4})) return EFFORT_ERR_ARG;
  DeviceGuard guard(m->dev);
  return launched(launch_fp8_matmul(m->w, m->ws, (int)m->I, (int)m->O, (const uint8_t*)x, x_stride, x_scales,
                                    x_scales_stride, rows, out_dtype, out, out_stride, (cudaStream_t)stream));
}

effort_status_t effort_fp8_get_info(effort_fp8_t m, int64_t* in_dim, int64_t* out_dim, size_t* device_bytes) {
  if (!m) return EFFORT_ERR_ARG;
  if (in_dim) *in_dim = m->I;
  if (out_dim) *out_dim = m->O;
  if (device_bytes) *device_bytes = m->buf.bytes;
  return EFFORT_OK;
}

effort_status_t effort_fp8_destroy(effort_fp8_t m) {
  if (!m) return EFFORT_ERR_ARG;
  {
    DeviceGuard guard(m->dev);
    m->buf.release();
  }
  delete m;
  return EFFORT_OK;
}

effort_status_t effort_moe_prepare(const effort_moe_weights_t* weights, void* stream, effort_moe_t* out_layer) {
  if (!out_layer) return EFFORT_ERR_ARG;
  *out_layer = nullptr;
  if (!weights) return EFFORT_ERR_ARG;
  const effort_moe_weights_t& a = *weights;
  const bool q = a.weight_kind == EFFORT_W_E4M3;
  if (a.n_experts < 1 || a.in_dim < 1 || a.hidden_dim < 1 || !a.w1 || !a.w3 || !a.w2) return EFFORT_ERR_ARG;
  if (!q && a.weight_kind != EFFORT_W_F16 && a.weight_kind != EFFORT_W_BF16) return EFFORT_ERR_ARG;
  if (q ? (!a.s1 || !a.s3 || !a.s2) : (a.s1 || a.s3 || a.s2)) return EFFORT_ERR_ARG;
  const size_t esz = q ? 1 : 2;
  if (!aligned(a.w1, esz) || !aligned(a.w3, esz) || !aligned(a.w2, esz) || !aligned(a.s1, 4) || !aligned(a.s3, 4) ||
      !aligned(a.s2, 4))
    return EFFORT_ERR_ARG;
  if (a.router && (!dtype_ok(a.router_dtype) || !aligned(a.router, dtype_size(a.router_dtype)))) return EFFORT_ERR_ARG;
  if (a.n_experts > EFFORT_MAX_EXPERTS || a.in_dim > EFFORT_MAX_IN_DIM || a.hidden_dim > EFFORT_MAX_IN_DIM)
    return EFFORT_ERR_UNSUPPORTED;
  const int E = a.n_experts, I = (int)a.in_dim, F = (int)a.hidden_dim, wk = (int)a.weight_kind;
  const int ke = k_per_block(wk);
  const int c13 = cdiv(2 * cdiv(F, 8), kGroupCores) * kGroupCores, c2 = cdiv(I, 8 * kGroupCores) * kGroupCores;
  const TileMat w13 = {nullptr, c13, cdiv(I, ke), (size_t)c13 * cdiv(I, ke) * kCoreBytes};
  const TileMat w2 = {nullptr, c2, cdiv(F, ke), (size_t)c2 * cdiv(F, ke) * kCoreBytes};
  const int bi = cdiv(I, kBlk), bf = cdiv(F, kBlk);
  const size_t scale_n = (size_t)E * bi * bf;
  // the scales as [row block][K block], rows of whole 16 bytes
  const size_t s13bytes = q ? align_up((size_t)E * bf * align4(bi) * 4, 256) : 0;
  const size_t s2bytes = q ? align_up((size_t)E * bi * align4(bf) * 4, 256) : 0;
  const int rpitch = (I + 7) / 8 * 8;  // the router's rows in whole 16 bytes
  const size_t rsz = a.router ? dtype_size(a.router_dtype) : 0, rbytes = align_up((size_t)E * rpitch * rsz, 256);
  const size_t nbytes = align_up((size_t)E * w2.nkb * sizeof(double2), 256);  // the column norms
  const size_t total = E * (w13.stride + w2.stride) + 2 * s13bytes + s2bytes + rbytes + nbytes + 256;
  if (!within_cap(total)) return EFFORT_ERR_NOMEM;
  effort_moe_s* h = new (std::nothrow) effort_moe_s();
  if (!h) return EFFORT_ERR_NOMEM;
  auto fail = [&](effort_status_t s) {
    cudaGetLastError();
    h->buf.release();
    delete h;
    return s;
  };
  effort_status_t st = device_sms(&h->sms);
  if (st != EFFORT_OK || cudaGetDevice(&h->dev) != cudaSuccess) return fail(EFFORT_ERR_CUDA);
  st = h->buf.alloc(total);
  if (st != EFFORT_OK) return fail(st);
  h->E = E;
  h->I = I;
  h->F = F;
  h->wk = wk;
  h->rdt = (int)a.router_dtype;
  h->rpitch = rpitch;
  char* b = (char*)h->buf.p;
  h->w13 = w13;
  h->w13.data = (const uint8_t*)b;
  b += E * w13.stride;
  h->w2 = w2;
  h->w2.data = (const uint8_t*)b;
  b += E * w2.stride;
  const float** dst[3] = {&h->s1, &h->s3, &h->s2};
  const float* src[3] = {a.s1, a.s3, a.s2};
  unsigned* status = (unsigned*)((char*)h->buf.p + total - 256);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemsetAsync(status, 0, 4, s);
  for (int i = 0; i < 3 && q; ++i) {
    *dst[i] = (const float*)b;
    if (e == cudaSuccess) e = launch_check_finite(src[i], scale_n, status, s);
    if (e == cudaSuccess) e = launch_turn_scales(src[i], E, i < 2 ? bi : bf, i < 2 ? bf : bi, (float*)b, s);
    b += i < 2 ? s13bytes : s2bytes;
  }
  if (a.router) {
    h->router = b;
    if (e == cudaSuccess) e = cudaMemsetAsync(b, 0, rbytes, s);
    if (e == cudaSuccess)
      e = cudaMemcpy2DAsync(b, rpitch * rsz, a.router, I * rsz, I * rsz, E, cudaMemcpyDeviceToDevice, s);
    b += rbytes;
  }
  h->bound = (const double2*)b;
  if (e == cudaSuccess) e = launch_moe_bounds(a.w1, a.w3, a.s1, a.s3, wk, E, I, F, (double2*)b, status, s);
  if (e == cudaSuccess)
    e = launch_tile_weights(wk, a.w1, E, I, F, (uint8_t*)h->w13.data, w13.cores, w13.nkb, w13.stride, 1, status, s);
  if (e == cudaSuccess)
    e = launch_tile_weights(wk, a.w3, E, I, F, (uint8_t*)h->w13.data, w13.cores, w13.nkb, w13.stride, 2, status, s);
  if (e == cudaSuccess)
    e = launch_tile_weights(wk, a.w2, E, F, I, (uint8_t*)h->w2.data, w2.cores, w2.nkb, w2.stride, 0, status, s);
  unsigned bad = 0;
  if (e == cudaSuccess) e = cudaMemcpyAsync(&bad, status, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return fail(EFFORT_ERR_CUDA);
  if (bad & 1) return fail(EFFORT_ERR_NONFINITE);
  h->spread = (bad & 2) != 0;
  *out_layer = h;
  return EFFORT_OK;
}

effort_status_t effort_moe_scratch_bytes(effort_moe_t h, int64_t n_tokens, int32_t top_k, size_t* bytes) {
  if (!h || !bytes || n_tokens < 0 || top_k < 1) return EFFORT_ERR_ARG;
  if (n_tokens > EFFORT_MAX_TOKENS || top_k > EFFORT_MAX_TOP_K) return EFFORT_ERR_UNSUPPORTED;
  *bytes = call_scratch(h, nullptr, nullptr, (int)n_tokens, top_k);
  return EFFORT_OK;
}

effort_status_t effort_moe_forward(effort_moe_t h, const void* x, effort_dtype_t x_dtype, int64_t x_stride,
                                   int64_t n_tokens, int32_t top_k, effort_gate_mode_t gate_mode, int32_t* ids,
                                   float* gates, void* out, effort_dtype_t out_dtype, int64_t out_stride, void* scratch,
                                   size_t scratch_bytes, void* stream) {
  if (!h || n_tokens < 0 || top_k < 1 || !dtype_ok(x_dtype) || !dtype_ok(out_dtype)) return EFFORT_ERR_ARG;
  if (gate_mode != EFFORT_GATE_SOFTMAX_OF_TOP && gate_mode != EFFORT_GATE_TOP_OF_SOFTMAX && gate_mode != EFFORT_GATE_GIVEN)
    return EFFORT_ERR_ARG;
  if (gate_mode != EFFORT_GATE_GIVEN && (!h->router || top_k > h->E)) return EFFORT_ERR_ARG;
  if (n_tokens > 0 && (!x || !ids || !gates || !out || !scratch)) return EFFORT_ERR_ARG;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(out, dtype_size(out_dtype)) || !aligned(ids, 4) || !aligned(gates, 4) ||
      !aligned(scratch, 256) || x_stride < h->I || out_stride < h->I)
    return EFFORT_ERR_ARG;
  if (n_tokens > EFFORT_MAX_TOKENS || top_k > EFFORT_MAX_TOP_K) return EFFORT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return EFFORT_OK;
  MoeCall c = {};
  if (scratch_bytes < call_scratch(h, nullptr, nullptr, (int)n_tokens, top_k)) return EFFORT_ERR_ARG;
  const int64_t xsz = (int64_t)dtype_size(x_dtype), osz = (int64_t)dtype_size(out_dtype);
  const Span sx = {x, n_tokens, x_stride * xsz, h->I * xsz}, so = {out, n_tokens, out_stride * osz, h->I * osz},
             si = {ids, 1, 0, n_tokens * top_k * 4}, sg = {gates, 1, 0, n_tokens * top_k * 4},
             ss = {scratch, 1, 0, (int64_t)scratch_bytes};
  const bool routes = gate_mode != EFFORT_GATE_GIVEN;  // the call writes ids and gates
  if (meet(so, si) || meet(so, sg) || meet(ss, so) || meet(ss, sx) || meet(ss, si) || meet(ss, sg) ||
      (routes && (meet(si, sg) || meet(si, sx) || meet(sg, sx))))
    return EFFORT_ERR_ARG;
  call_scratch(h, &c, (char*)scratch, (int)n_tokens, top_k);
  DeviceGuard guard(h->dev);
  c.w13 = h->w13;
  c.w2 = h->w2;
  c.s1 = h->s1;
  c.s3 = h->s3;
  c.s2 = h->s2;
  c.bound = h->bound;
  c.spread = h->spread;
  c.nsb13 = cdiv(h->F, kBlk);
  c.nsb2 = cdiv(h->I, kBlk);
  c.router = h->router;
  c.rdt = h->rdt;
  c.rpitch = h->rpitch;
  c.wk = h->wk;
  c.n_experts = h->E;
  c.I = (int)h->I;
  c.F = (int)h->F;
  c.x = x;
  c.xdt = x_dtype;
  c.xstride = x_stride;
  c.n_tokens = (int)n_tokens;
  c.top_k = top_k;
  c.gate_mode = gate_mode;
  c.ids = ids;
  c.gates = gates;
  c.out = out;
  c.odt = out_dtype;
  c.ostride = out_stride;
  return launched(launch_moe(c, h->sms, (cudaStream_t)stream));
}

effort_status_t effort_moe_get_info(effort_moe_t h, int32_t* n_experts, int64_t* in_dim, int64_t* hidden_dim,
                                    size_t* device_bytes) {
  if (!h) return EFFORT_ERR_ARG;
  if (n_experts) *n_experts = h->E;
  if (in_dim) *in_dim = h->I;
  if (hidden_dim) *hidden_dim = h->F;
  if (device_bytes) *device_bytes = h->buf.bytes;
  return EFFORT_OK;
}

effort_status_t effort_moe_destroy(effort_moe_t h) {
  if (!h) return EFFORT_ERR_ARG;
  {
    DeviceGuard guard(h->dev);
    h->buf.release();
  }
  delete h;
  return EFFORT_OK;
}

}  // extern "C"
