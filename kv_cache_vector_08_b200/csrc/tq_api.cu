// C ABI of libtq: argument checking, context construction and kernel dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "common.cuh"
#include "kernels.cuh"

namespace tq {

namespace {
thread_local std::string g_error;
std::atomic<uint64_t> g_launches{0};
std::atomic<uint64_t> g_wait_ns{2000000000ull};
std::atomic<int> g_stall{0};
std::atomic<int> g_fail_alloc{-1};     // index of the tq_init allocation to fail (-1: none)
std::atomic<int> g_alloc_count{0};
}  // namespace

uint64_t pipeline_wait_ns() { return g_wait_ns.load(std::memory_order_relaxed); }
bool debug_stall() { return g_stall.load(std::memory_order_relaxed) != 0; }

cudaError_t dev_alloc(void** p, size_t bytes) {
  const int i = g_alloc_count.fetch_add(1, std::memory_order_relaxed);
  if (i == g_fail_alloc.load(std::memory_order_relaxed)) {
    *p = nullptr;
    return cudaErrorMemoryAllocation;
  }
  return cudaMalloc(p, bytes);
}

// NVTX range around each entry point (a no-op unless a profiler is attached).
struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

void set_error(const std::string& msg) { g_error = msg; }

int fail(int code, const std::string& msg) {
  g_error = msg;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  g_error = std::string(what) + ": " + cudaGetErrorString(e);
  return TQ_ERR_CUDA;
}

void count_launch(uint64_t n) { g_launches.fetch_add(n, std::memory_order_relaxed); }

int check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, what);
  return TQ_OK;
}

namespace {

int check_device(const tq_ctx* ctx) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev != ctx->device) return fail(TQ_ERR_INVALID_ARG, "context belongs to another CUDA device than the current one");
  return TQ_OK;
}

bool bad_dtype(int t) { return t != TQ_DTYPE_F32 && t != TQ_DTYPE_BF16 && t != TQ_DTYPE_F16; }
size_t elem_size(int t) { return t == TQ_DTYPE_F32 ? 4 : 2; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_packed(const tq_ctx* ctx, const tq_packed* pk, const char* name) {
  if (!pk) return fail(TQ_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (!pk->codes || !pk->norm) return fail(TQ_ERR_INVALID_ARG, std::string(name) + ": codes/norm pointer is NULL");
  if (ctx->mode == TQ_MODE_PROD && !pk->rnorm)
    return fail(TQ_ERR_INVALID_ARG, std::string(name) + ": rnorm is required for a prod-mode context");
  if (pk->cap < 0) return fail(TQ_ERR_INVALID_ARG, std::string(name) + ": negative capacity");
  if (!aligned(pk->codes, 16)) return fail(TQ_ERR_UNSUPPORTED, std::string(name) + ": codes must be 16-byte aligned");
  return TQ_OK;
}

int alloc_copy(float** dst, const std::vector<double>& src) {
  std::vector<float> f(src.size());
  for (size_t i = 0; i < src.size(); ++i) f[i] = (float)src[i];
  cudaError_t e = dev_alloc(reinterpret_cast<void**>(dst), f.size() * sizeof(float));
  if (e != cudaSuccess) {
    *dst = nullptr;
    return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  }
  e = cudaMemcpy(*dst, f.data(), f.size() * sizeof(float), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(params)");
  return TQ_OK;
}

std::vector<double> transpose(const std::vector<double>& a, int rows, int cols) {
  std::vector<double> t((size_t)rows * cols);
  for (int i = 0; i < rows; ++i)
    for (int j = 0; j < cols; ++j) t[(size_t)j * rows + i] = a[(size_t)i * cols + j];
  return t;
}

// bf16 / fp16 splits of the tensor-core operands: Pi = hi + mid + lo (bf16, ~24 bits),
// 16*M = hi + lo (fp16, ~22 bits); each split row-major [d][d].
int alloc_splits(tq_ctx* c) {
  const HostParams& h = c->host;
  const int d = c->lay.d;
  const size_t nn = (size_t)d * d;
  std::vector<__nv_bfloat16> pis(3 * nn);
  for (size_t i = 0; i < nn; ++i) {
    double v = h.Pi[i];
    __nv_bfloat16 a = __float2bfloat16_rn((float)v);
    double r1 = v - (double)__bfloat162float(a);
    __nv_bfloat16 b = __float2bfloat16_rn((float)r1);
    double r2 = r1 - (double)__bfloat162float(b);
    pis[i] = a;
    pis[nn + i] = b;
    pis[2 * nn + i] = __float2bfloat16_rn((float)r2);
  }
  cudaError_t e = dev_alloc(&c->Pi_split, pis.size() * sizeof(__nv_bfloat16));
  if (e != cudaSuccess) return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  e = cudaMemcpy(c->Pi_split, pis.data(), pis.size() * sizeof(__nv_bfloat16), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(Pi splits)");
  if (c->mode == TQ_MODE_PROD) {
    std::vector<__half> ms(2 * nn);
    for (size_t i = 0; i < nn; ++i) {
      double v = 16.0 * h.M[i];
      __half a = __float2half_rn((float)v);
      ms[i] = a;
      ms[nn + i] = __float2half_rn((float)(v - (double)__half2float(a)));
    }
    e = dev_alloc(&c->M_split, ms.size() * sizeof(__half));
    if (e != cudaSuccess) return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
    e = cudaMemcpy(c->M_split, ms.data(), ms.size() * sizeof(__half), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(M splits)");
  }
  return TQ_OK;
}

// Dequantize operands (d <= 128): B[n][k] = 16 A[k][n] * scale as fp16 hi + lo, [2][N][d_pad],
// for A = Pi (plain reconstruction) and A = S with scale sqrt(pi/2)/m (QJL term).
int alloc_dequant_operand(void** dst, const std::vector<double>& A, int d, int d_pad, double scale) {
  const int K = d_pad, N = 16 * ((d + 15) / 16);
  std::vector<__half> b((size_t)2 * N * K, __float2half(0.f));
  for (int n = 0; n < d; ++n)
    for (int k = 0; k < d; ++k) {
      const double v = 16.0 * scale * A[(size_t)k * d + n];
      const __half h = __float2half_rn((float)v);
      b[(size_t)n * K + k] = h;
      b[(size_t)N * K + (size_t)n * K + k] = __float2half_rn((float)(v - (double)__half2float(h)));
    }
  cudaError_t e = dev_alloc(dst, b.size() * sizeof(__half));
  if (e != cudaSuccess) return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  e = cudaMemcpy(*dst, b.data(), b.size() * sizeof(__half), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(dequantize operand)");
  return TQ_OK;
}

// Projection operands of the workspace quantize path: 16 Pi and 16 M as fp16 hi + lo,
// [2][d_pad][K] (K = 64 ceil(d/64)), zero padded.
int alloc_projection(void** dst, const std::vector<double>& A, int d, int d_pad) {
  const int K = 64 * ((d + 63) / 64);
  std::vector<__half> b((size_t)2 * d_pad * K, __float2half(0.f));
  for (int n = 0; n < d; ++n)
    for (int k = 0; k < d; ++k) {
      const double v = 16.0 * A[(size_t)n * d + k];
      const __half h = __float2half_rn((float)v);
      b[(size_t)n * K + k] = h;
      b[(size_t)d_pad * K + (size_t)n * K + k] = __float2half_rn((float)(v - (double)__half2float(h)));
    }
  cudaError_t e = dev_alloc(dst, b.size() * sizeof(__half));
  if (e != cudaSuccess) return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  e = cudaMemcpy(*dst, b.data(), b.size() * sizeof(__half), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(projection operand)");
  return TQ_OK;
}

void release(tq_ctx* c) {
  if (!c) return;
  cudaFree(c->Pi16);
  cudaFree(c->M16);
  cudaFree(c->PiT_f16);
  cudaFree(c->ST_f16);
  cudaFree(c->Pi_split);
  cudaFree(c->M_split);
  cudaFree(c->dev_err);
  cudaFree(c->Pi);
  cudaFree(c->PiT);
  cudaFree(c->ST);
  delete c;
}

// Factor in [1, 2) for which the positive levels times the factor are closest to fp16 numbers (the
// smallest maximum of their relative rounding errors over 2^16 steps; up to 8 levels, where the first
// try alone would leave up to 2^-11).
float level_scale(const std::vector<double>& c) {
  float best = 1.f;
  double best_err = 1e300;
  const size_t half = c.size() / 2;
  for (int i = 0; i < 1 << 16; ++i) {
    const float f = 1.f + (float)i / (1 << 16);
    double err = 0.0;
    for (size_t j = half; j < c.size() && err < best_err; ++j) {
      const double v = c[j] * f;
      err = std::max(err, std::fabs((double)__half2float(__float2half_rn((float)v)) - v) / v);
    }
    if (err < best_err) {
      best_err = err;
      best = f;
    }
  }
  return best;
}

int check_args_common(int d, int bits, int mode) {
  if (mode != TQ_MODE_PROD && mode != TQ_MODE_MSE) return fail(TQ_ERR_INVALID_ARG, "mode must be TQ_MODE_PROD or TQ_MODE_MSE");
  if (d < 3 || d > 4096) return fail(TQ_ERR_UNSUPPORTED, "d must be in [3, 4096]");
  if (mode == TQ_MODE_PROD && (bits < 2 || bits > 5)) return fail(TQ_ERR_UNSUPPORTED, "prod mode needs bits in [2, 5]");
  if (mode == TQ_MODE_MSE && (bits < 1 || bits > 4)) return fail(TQ_ERR_UNSUPPORTED, "MSE mode needs bits in [1, 4]");
  return TQ_OK;
}

}  // namespace

// Every argument check of tq_decode_attention except the workspace size (shared with
// tq_decode_attention_static, which checks its own scratch size after these).
int check_decode_args(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                      const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                      const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len, const void* out,
                      int page, bool any_dtype) {
  if (!kctx || !vctx || !group_off || !kcache || !vcache) return fail(TQ_ERR_INVALID_ARG, "NULL argument");
  if (ngroups < 1 || ngroups > 4) return fail(TQ_ERR_UNSUPPORTED, "ngroups must be in [1, 4]");
  if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_len < 0) return fail(TQ_ERR_INVALID_ARG, "bad sizes");
  if (Hq % Hkv != 0) return fail(TQ_ERR_INVALID_ARG, "Hq must be a multiple of Hkv");
  if (any_dtype ? bad_dtype(q_dtype) : q_dtype != TQ_DTYPE_F32 && q_dtype != TQ_DTYPE_BF16)
    return fail(TQ_ERR_INVALID_ARG, any_dtype ? "q_dtype must be F32, BF16 or F16" : "q_dtype must be F32 or BF16");
  if (group_off[0] != 0 || group_off[ngroups] != D) return fail(TQ_ERR_INVALID_ARG, "group_off must span [0, D]");
  if (B == 0) return TQ_OK;
  if (!q || !seq_lens || !out) return fail(TQ_ERR_INVALID_ARG, "NULL q, seq_lens or out");
  for (int g = 0; g < ngroups; ++g) {
    const tq_ctx* kc = kctx[g];
    const tq_ctx* vc = vctx[g];
    if (!kc || !vc) return fail(TQ_ERR_INVALID_ARG, "NULL context");
    int w = group_off[g + 1] - group_off[g];
    if (w <= 0) return fail(TQ_ERR_INVALID_ARG, "group_off must be increasing");
    if (kc->mode != TQ_MODE_PROD || vc->mode != TQ_MODE_MSE)
      return fail(TQ_ERR_INVALID_ARG, "key contexts must be prod mode, value contexts MSE mode");
    if (kc->lay.d != w || vc->lay.d != w) return fail(TQ_ERR_INVALID_ARG, "context dimension differs from its group width");
    int r = check_packed(kc, &kcache[g], "kcache");
    if (r != TQ_OK) return r;
    if ((r = check_packed(vc, &vcache[g], "vcache")) != TQ_OK) return r;
    // contiguous caches hold every (sequence, kv head, token) slot; paged ones at least one page
    int64_t need = page > 0 ? (int64_t)Hkv * page : (int64_t)B * Hkv * max_len;
    if (kcache[g].cap < need || vcache[g].cap < need)
      return fail(TQ_ERR_INVALID_ARG, page > 0 ? "cache capacity below one page (Hkv*page_tokens)"
                                               : "cache capacity below B*Hkv*max_len");
    if ((r = check_device(kc)) != TQ_OK) return r;
  }
  return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

const char* tq_last_error(void) { return g_error.c_str(); }

int tq_channel_perm_by_score(const float* score, int D, int w0, int32_t* perm) {
  if (!score || !perm || D <= 0 || w0 < 0 || w0 > D) return fail(TQ_ERR_INVALID_ARG, "bad channel permutation arguments");
  std::vector<int> order(D);
  for (int i = 0; i < D; ++i) order[i] = i;
  // the w0 highest scores (ties to the lower channel) form the first group
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return score[a] > score[b]; });
  std::vector<char> first(D, 0);
  for (int i = 0; i < w0; ++i) first[order[i]] = 1;
  int p = 0;
  for (int i = 0; i < D; ++i)
    if (first[i]) perm[p++] = i;
  for (int i = 0; i < D; ++i)
    if (!first[i]) perm[p++] = i;
  return TQ_OK;
}

int tq_debug_set_wait_limit(uint64_t ns) {
  g_wait_ns.store(ns, std::memory_order_relaxed);
  return TQ_OK;
}

int tq_debug_inject_stall(int on) {
  g_stall.store(on ? 1 : 0, std::memory_order_relaxed);
  return TQ_OK;
}

int tq_debug_fail_alloc(int index) {
  g_alloc_count.store(0, std::memory_order_relaxed);
  g_fail_alloc.store(index, std::memory_order_relaxed);
  return TQ_OK;
}

uint64_t tq_kernel_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int tq_host_params(int d, int bits, uint64_t seed, int mode, double* Pi, double* S, double* centroids,
                   double* boundaries) {
  int r = check_args_common(d, bits, mode);
  if (r != TQ_OK) return r;
  HostParams p;
  if (!build_params(d, bits, seed, mode, &p)) return fail(TQ_ERR_INVALID_ARG, "bad parameters");
  if (Pi) std::memcpy(Pi, p.Pi.data(), p.Pi.size() * sizeof(double));
  if (S && mode == TQ_MODE_PROD) std::memcpy(S, p.S.data(), p.S.size() * sizeof(double));
  if (centroids) std::memcpy(centroids, p.centroids.data(), p.centroids.size() * sizeof(double));
  if (boundaries) std::memcpy(boundaries, p.boundaries.data(), p.boundaries.size() * sizeof(double));
  return TQ_OK;
}

int tq_init(tq_ctx** out, int d, int bits, uint64_t seed, int mode) {
  Range range_("tq_init");
  if (!out) return fail(TQ_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  int r = check_args_common(d, bits, mode);
  if (r != TQ_OK) return r;
  tq_ctx* c = new (std::nothrow) tq_ctx();
  if (!c) return fail(TQ_ERR_ALLOC, "host allocation failed");
  cudaError_t e = cudaGetDevice(&c->device);
  if (e != cudaSuccess) {
    delete c;
    return cuda_fail(e, "cudaGetDevice");
  }
  if (!build_params(d, bits, seed, mode, &c->host)) {
    delete c;
    return fail(TQ_ERR_INVALID_ARG, "bad parameters");
  }
  const HostParams& h = c->host;
  c->mode = mode;
  c->bits = bits;
  c->m = h.m;
  Layout& L = c->lay;
  L.d = d;
  L.k = h.k;
  L.d_pad = ((d + 31) / 32) * 32;
  L.planes = h.k + (mode == TQ_MODE_PROD ? 1 : 0);
  L.code_bytes = L.planes * L.d_pad / 8;
  Codebook& cb = c->cb;
  cb.K = 1 << h.k;
  for (int j = 0; j < kMaxLevels; ++j) {
    cb.c[j] = j < cb.K ? (float)h.centroids[j] : 0.f;
    cb.t[j] = j < cb.K - 1 ? (float)h.boundaries[j] : INFINITY;
  }
  for (int code = 0; code < kMaxLevels; ++code) cb.cc[code] = code < cb.K ? cb.c[code_index(code, h.k)] : 0.f;
  c->lev_scale = level_scale(h.centroids);
  c->sqrt_pi_over_2_over_m = mode == TQ_MODE_PROD ? (float)(std::sqrt(M_PI / 2.0) / h.m) : 0.f;
  for (int j = 0; j < h.m; ++j) {
    double r = 0.0;
    for (int i = 0; i < d; ++i) r += h.S[(size_t)j * d + i] * h.S[(size_t)j * d + i];
    c->s_rowmax = std::max(c->s_rowmax, (float)(std::sqrt(r) * (1.0 + 1e-6)));
  }
  if ((r = alloc_copy(&c->Pi, h.Pi)) != TQ_OK || (r = alloc_copy(&c->PiT, transpose(h.Pi, d, d))) != TQ_OK) {
    release(c);
    return r;
  }
  if (mode == TQ_MODE_PROD) {
    if ((r = alloc_copy(&c->ST, transpose(h.S, h.m, d))) != TQ_OK) {
      release(c);
      return r;
    }
  }
  if (d == 64 || d == 128) {
    if ((r = alloc_splits(c)) != TQ_OK) {
      release(c);
      return r;
    }
  }
  if (d <= 128 && ((r = alloc_dequant_operand(&c->PiT_f16, h.Pi, d, L.d_pad, 1.0)) != TQ_OK ||
                    (mode == TQ_MODE_PROD &&
                     (r = alloc_dequant_operand(&c->ST_f16, h.S, d, L.d_pad, std::sqrt(M_PI / 2.0) / h.m)) != TQ_OK))) {
    release(c);
    return r;
  }
  if ((r = alloc_projection(&c->Pi16, h.Pi, d, L.d_pad)) != TQ_OK ||
      (mode == TQ_MODE_PROD && (r = alloc_projection(&c->M16, h.M, d, L.d_pad)) != TQ_OK)) {
    release(c);
    return r;
  }
  e = dev_alloc(reinterpret_cast<void**>(&c->dev_err), sizeof(int));
  if (e != cudaSuccess) {
    release(c);
    return fail(TQ_ERR_ALLOC, std::string("cudaMalloc: ") + cudaGetErrorString(e));
  }
  e = cudaMemset(c->dev_err, 0, sizeof(int));
  if (e != cudaSuccess) {
    release(c);
    return cuda_fail(e, "cudaMemset(error word)");
  }
  *out = c;
  return TQ_OK;
}

int tq_get_device_error(const tq_ctx* ctx, int* code) {
  if (!ctx || !code) return fail(TQ_ERR_INVALID_ARG, "NULL argument");
  int v = 0;
  cudaError_t e = cudaMemcpy(&v, ctx->dev_err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy(error word)");
  *code = v;
  if (v != 0) {
    e = cudaMemset(ctx->dev_err, 0, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemset(error word)");
  }
  return TQ_OK;
}

void tq_free(tq_ctx* ctx) { release(ctx); }

int tq_get_info(const tq_ctx* ctx, tq_info* info) {
  if (!ctx || !info) return fail(TQ_ERR_INVALID_ARG, "NULL argument");
  info->d = ctx->lay.d;
  info->bits = ctx->bits;
  info->k = ctx->lay.k;
  info->m = ctx->m;
  info->mode = ctx->mode;
  info->planes = ctx->lay.planes;
  info->d_pad = ctx->lay.d_pad;
  info->code_bytes = ctx->lay.code_bytes;
  info->seed = ctx->host.seed;
  return TQ_OK;
}

int tq_get_params(const tq_ctx* ctx, double* Pi, double* S, double* centroids, double* boundaries) {
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  const HostParams& h = ctx->host;
  if (Pi) std::memcpy(Pi, h.Pi.data(), h.Pi.size() * sizeof(double));
  if (S && ctx->mode == TQ_MODE_PROD) std::memcpy(S, h.S.data(), h.S.size() * sizeof(double));
  if (centroids) std::memcpy(centroids, h.centroids.data(), h.centroids.size() * sizeof(double));
  if (boundaries) std::memcpy(boundaries, h.boundaries.data(), h.boundaries.size() * sizeof(double));
  return TQ_OK;
}

size_t tq_quantize_workspace_size(const tq_ctx* ctx, int x_dtype, int64_t n, int64_t ld) {
  if (!ctx || n < 0) return 0;
  if (n == 0 || quantize_tc_applies(ctx, x_dtype, n, ld)) return 0;
  return quantize_gen_workspace(ctx, n);
}

static int quantize_common(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const int32_t* cols,
                           const tq_packed* dst, const int64_t* dst_slot, void* workspace, size_t ws_bytes,
                           tq_stream_t stream) {
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "n < 0");
  if (n > 0 && !x) return fail(TQ_ERR_INVALID_ARG, "x is NULL");
  if (ld < ctx->lay.d) return fail(TQ_ERR_INVALID_ARG, "ld < d");
  if (x_dtype != TQ_DTYPE_F32 && x_dtype != TQ_DTYPE_BF16 && x_dtype != TQ_DTYPE_F16)
    return fail(TQ_ERR_INVALID_ARG, "x_dtype must be TQ_DTYPE_F32, BF16 or F16");
  int r = check_packed(ctx, dst, "dst");
  if (r != TQ_OK) return r;
  if (!dst_slot && n > dst->cap) return fail(TQ_ERR_INVALID_ARG, "n exceeds dst->cap");
  if ((r = check_device(ctx)) != TQ_OK) return r;
  if (n == 0) return TQ_OK;
  if (cols)
    return launch_quantize_gen(ctx, x, x_dtype, n, ld, cols, dst, dst_slot, workspace, ws_bytes, (cudaStream_t)stream);
  return launch_quantize(ctx, x, x_dtype, n, ld, dst, dst_slot, workspace, ws_bytes, (cudaStream_t)stream);
}

int tq_quantize_kv(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const tq_packed* dst,
                   const int64_t* dst_slot, void* workspace, size_t ws_bytes, tq_stream_t stream) {
  Range range_("tq_quantize_kv");
  return quantize_common(ctx, x, x_dtype, n, ld, nullptr, dst, dst_slot, workspace, ws_bytes, stream);
}

size_t tq_quantize_cols_workspace_size(const tq_ctx* ctx, int64_t n) {
  if (!ctx || n <= 0) return 0;
  return quantize_gen_workspace(ctx, n);
}

int tq_quantize_kv_cols(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const int32_t* cols,
                        const tq_packed* dst, const int64_t* dst_slot, void* workspace, size_t ws_bytes,
                        tq_stream_t stream) {
  Range range_("tq_quantize_kv_cols");
  if (!cols) return fail(TQ_ERR_INVALID_ARG, "cols is NULL");
  return quantize_common(ctx, x, x_dtype, n, ld, cols, dst, dst_slot, workspace, ws_bytes, stream);
}

static int dequantize_common(const tq_ctx* ctx, const tq_packed* src, const int64_t* src_slot, int64_t n, float* out,
                             int64_t ld, bool qjl, tq_stream_t stream) {
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, "n < 0");
  if (n > 0 && !out) return fail(TQ_ERR_INVALID_ARG, "out is NULL");
  if (ld < ctx->lay.d) return fail(TQ_ERR_INVALID_ARG, "ld < d");
  if (qjl && ctx->mode != TQ_MODE_PROD) return fail(TQ_ERR_INVALID_ARG, "the QJL reconstruction needs a prod-mode context");
  int r = check_packed(ctx, src, "src");
  if (r != TQ_OK) return r;
  if (!src_slot && n > src->cap) return fail(TQ_ERR_INVALID_ARG, "n exceeds src->cap");
  if ((r = check_device(ctx)) != TQ_OK) return r;
  return launch_dequantize_tc(ctx, src, src_slot, n, out, ld, qjl, (cudaStream_t)stream);
}

int tq_dequantize(const tq_ctx* ctx, const tq_packed* src, const int64_t* src_slot, int64_t n, float* out,
                  int64_t ld, tq_stream_t stream) {
  Range range_("tq_dequantize");
  return dequantize_common(ctx, src, src_slot, n, out, ld, false, stream);
}

int tq_dequantize_qjl(const tq_ctx* ctx, const tq_packed* src, const int64_t* src_slot, int64_t n, float* out,
                      int64_t ld, tq_stream_t stream) {
  Range range_("tq_dequantize_qjl");
  return dequantize_common(ctx, src, src_slot, n, out, ld, true, stream);
}

int tq_prepare_queries(const tq_ctx* ctx, const float* q, int64_t nq, int64_t ld, float* out, tq_stream_t stream) {
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  if (nq < 0) return fail(TQ_ERR_INVALID_ARG, "nq < 0");
  if (nq > 0 && (!q || !out)) return fail(TQ_ERR_INVALID_ARG, "NULL q or out");
  if (ld < ctx->lay.d) return fail(TQ_ERR_INVALID_ARG, "ld < d");
  int r = check_device(ctx);
  if (r != TQ_OK) return r;
  return launch_prepare_queries(ctx, q, TQ_DTYPE_F32, nq, ld, out, ctx->lay.d + ctx->m, (cudaStream_t)stream);
}

size_t tq_attn_logits_workspace_size(const tq_ctx* ctx, int64_t nq) {
  if (!ctx || nq < 0) return 0;
  return logits_mma_workspace(nq, ctx->lay.d);
}

int tq_attn_logits(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* keys, int64_t n, float* logits,
                   void* workspace, size_t ws_bytes, tq_stream_t stream) {
  Range range_("tq_attn_logits");
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  if (nq < 0 || n < 0) return fail(TQ_ERR_INVALID_ARG, "negative size");
  if (nq > 0 && (!q || !logits) && n > 0) return fail(TQ_ERR_INVALID_ARG, "NULL q or logits");
  int r = check_packed(ctx, keys, "keys");
  if (r != TQ_OK) return r;
  if (n > keys->cap) return fail(TQ_ERR_INVALID_ARG, "n exceeds keys->cap");
  size_t need = tq_attn_logits_workspace_size(ctx, nq);
  if (need > 0 && (!workspace || ws_bytes < need)) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  if ((r = check_device(ctx)) != TQ_OK) return r;
  if (nq == 0 || n == 0) return TQ_OK;
  return launch_logits(ctx, q, nq, keys, n, logits, workspace, (cudaStream_t)stream);
}

size_t tq_decode_workspace_size(int B, int Hq, int Hkv, int D, int ngroups, int64_t max_len) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || ngroups <= 0 || max_len < 0) return 0;
  return decode_workspace_bytes(B, Hq, Hkv, D, ngroups, max_len, D);
}

int tq_decode_attention_ex(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                           const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                           const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len, float scale,
                           float* out, const tq_decode_opts* opts, void* workspace, size_t ws_bytes,
                           tq_stream_t stream) {
  Range range_("tq_decode_attention");
  const int32_t* perm = opts ? opts->channel_perm : nullptr;
  const int32_t* table = opts ? opts->block_table : nullptr;
  const int page = table ? opts->page_tokens : 0;
  if (table && (page <= 0 || page % 64 != 0 || max_len % page != 0))
    return fail(TQ_ERR_INVALID_ARG, "page_tokens must be a positive multiple of 64 that divides max_len");
  int r = check_decode_args(kctx, vctx, group_off, ngroups, q, q_dtype, kcache, vcache, seq_lens, B, Hq, Hkv, D,
                            max_len, out, page);
  if (r != TQ_OK) return r;
  if (B == 0) return TQ_OK;
  size_t need = tq_decode_workspace_size(B, Hq, Hkv, D, ngroups, max_len);
  if (!workspace || ws_bytes < need) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  return launch_decode(kctx, vctx, group_off, ngroups, perm, table, page, q, q_dtype, kcache, vcache, seq_lens, B, Hq,
                       Hkv, D, max_len, scale, out, workspace, (cudaStream_t)stream);
}

int tq_decode_attention(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                        const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                        const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len, float scale,
                        float* out, void* workspace, size_t ws_bytes, tq_stream_t stream) {
  return tq_decode_attention_ex(kctx, vctx, group_off, ngroups, q, q_dtype, kcache, vcache, seq_lens, B, Hq, Hkv, D,
                                max_len, scale, out, nullptr, workspace, ws_bytes, stream);
}

size_t tq_search_workspace_size(const tq_ctx* ctx, int64_t nq, int64_t N, int k) {
  if (!ctx || nq < 0 || N < 0 || k < 1) return 0;
  return search_tc_workspace(ctx, nq, N, k);
}

int tq_search_topk(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* db, int64_t N, int k,
                   float* scores, int64_t* ids, void* workspace, size_t ws_bytes, tq_stream_t stream) {
  Range range_("tq_search_topk");
  if (!ctx) return fail(TQ_ERR_INVALID_ARG, "ctx is NULL");
  if (ctx->mode != TQ_MODE_PROD) return fail(TQ_ERR_INVALID_ARG, "search needs a prod-mode context");
  if (nq < 0 || N < 1) return fail(TQ_ERR_INVALID_ARG, "bad sizes");
  if (k < 1 || k > 64 || k > N) return fail(TQ_ERR_UNSUPPORTED, "k must be in [1, min(64, N)]");
  int r = check_packed(ctx, db, "db");
  if (r != TQ_OK) return r;
  if (N > db->cap) return fail(TQ_ERR_INVALID_ARG, "N exceeds db->cap");
  if (nq > 0 && (!q || !scores || !ids)) return fail(TQ_ERR_INVALID_ARG, "NULL q, scores or ids");
  size_t need = tq_search_workspace_size(ctx, nq, N, k);
  if (!workspace || ws_bytes < need) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  if ((r = check_device(ctx)) != TQ_OK) return r;
  return launch_search(ctx, q, nq, db, N, k, scores, ids, workspace, (cudaStream_t)stream);
}

int tq_rope(const tq_rope_tensor* tensors, int ntensors, int dtype, int64_t n, int D, int rot, const double* freq,
            const void* pos, int pos_bits, double factor, int flags, tq_stream_t stream) {
  Range range_("tq_rope");
  if (!tensors || ntensors < 1 || ntensors > 2) return fail(TQ_ERR_INVALID_ARG, "tq_rope: one or two tensors");
  if (bad_dtype(dtype)) return fail(TQ_ERR_INVALID_ARG, "tq_rope: dtype must be F32, BF16 or F16");
  if (n < 0 || D <= 0) return fail(TQ_ERR_INVALID_ARG, "tq_rope: bad sizes");
  if (rot < 2 || rot > D || rot % 2 != 0) return fail(TQ_ERR_INVALID_ARG, "tq_rope: rot must be even and in [2, D]");
  if (D > 4096) return fail(TQ_ERR_UNSUPPORTED, "tq_rope: D must be at most 4096");
  if (pos_bits != 32 && pos_bits != 64) return fail(TQ_ERR_INVALID_ARG, "tq_rope: pos_bits must be 32 or 64");
  if (flags & ~(TQ_ROPE_INTERLEAVED | TQ_ROPE_TRANSPOSE)) return fail(TQ_ERR_INVALID_ARG, "tq_rope: unknown flags");
  for (int i = 0; i < ntensors; ++i) {
    if (tensors[i].heads < 0) return fail(TQ_ERR_INVALID_ARG, "tq_rope: negative head count");
    if (n == 0 || tensors[i].heads == 0) continue;
    if (!tensors[i].x || !tensors[i].out) return fail(TQ_ERR_INVALID_ARG, "tq_rope: NULL tensor");
    if (!aligned(tensors[i].x, elem_size(dtype)) || !aligned(tensors[i].out, elem_size(dtype)))
      return fail(TQ_ERR_UNSUPPORTED, "tq_rope: a tensor is not aligned to its element");
  }
  if (n == 0) return TQ_OK;
  if (!freq || !pos) return fail(TQ_ERR_INVALID_ARG, "tq_rope: NULL freq or pos");
  return launch_rope(tensors, ntensors, dtype, n, D, rot, freq, pos, pos_bits, factor, flags, (cudaStream_t)stream);
}

int tq_rope_frequencies(int rot, double base, const tq_rope_scaling* s, double* freq, double* factor_out) {
  if (!freq || !factor_out) return fail(TQ_ERR_INVALID_ARG, "tq_rope_frequencies: NULL output");
  if (rot < 2 || rot % 2 != 0 || !(base > 1.0)) return fail(TQ_ERR_INVALID_ARG, "tq_rope_frequencies: rot must be even, base above 1");
  if (s) {
    if (s->kind < TQ_ROPE_SCALE_NONE || s->kind > TQ_ROPE_SCALE_YARN)
      return fail(TQ_ERR_INVALID_ARG, "tq_rope_frequencies: unknown scaling");
    if (s->kind != TQ_ROPE_SCALE_NONE && !(s->factor > 0.0))
      return fail(TQ_ERR_INVALID_ARG, "tq_rope_frequencies: factor must be positive");
    if ((s->kind == TQ_ROPE_SCALE_BANDS || s->kind == TQ_ROPE_SCALE_YARN) &&
        (!(s->original_len > 0.0) || !(s->low < s->high) || !(s->low > 0.0)))
      return fail(TQ_ERR_INVALID_ARG, "tq_rope_frequencies: needs original_len > 0 and 0 < low < high");
  }
  return rope_frequencies(rot, base, s, freq, factor_out);
}

int tq_page_bounds(const void* k, int64_t n, int dtype, int64_t k_token, int64_t k_head, const int32_t* cu_new,
                   const int32_t* start, int B, int Hkv, int D, int64_t max_new, const int32_t* block_table,
                   int page_tokens, int max_pages, void* bounds, int64_t npages, tq_stream_t stream) {
  Range range_("tq_page_bounds");
  if (bad_dtype(dtype)) return fail(TQ_ERR_INVALID_ARG, "tq_page_bounds: dtype must be F32, BF16 or F16");
  if (n < 0 || B < 0 || Hkv <= 0 || D <= 0 || max_new < 0 || page_tokens <= 0 || max_pages < 0 || npages < 0)
    return fail(TQ_ERR_INVALID_ARG, "tq_page_bounds: bad sizes");
  if (D > 256 || B > 65535 || Hkv > 65535)
    return fail(TQ_ERR_UNSUPPORTED, "tq_page_bounds: D must be at most 256, B and Hkv at most 65535");
  if (n == 0 || B == 0 || max_new == 0 || max_pages == 0 || npages == 0) return TQ_OK;
  if (!k || !cu_new || !start || !block_table || !bounds) return fail(TQ_ERR_INVALID_ARG, "tq_page_bounds: NULL argument");
  if (!aligned(k, elem_size(dtype)) || !aligned(bounds, elem_size(dtype)))
    return fail(TQ_ERR_UNSUPPORTED, "tq_page_bounds: a pointer is not aligned to its element");
  return launch_page_bounds(k, n, dtype, k_token, k_head, cu_new, start, B, Hkv, D, max_new, block_table, page_tokens,
                            max_pages, bounds, npages, (cudaStream_t)stream);
}

// Limits that the sparse and tree calls share with the decode launches.
static int check_cache_shape(int64_t pairs, int64_t rows, int64_t max_len, const char* what) {
  if (max_len > (int64_t)1 << 30) return fail(TQ_ERR_UNSUPPORTED, std::string(what) + ": max_len above 2^30");
  if (pairs > 65535 || rows > (int64_t)1 << 24)
    return fail(TQ_ERR_UNSUPPORTED, std::string(what) + ": more than 65535 (sequence, kv head, 4 query heads) blocks or "
                                                        "2^24 query rows");
  return TQ_OK;
}

static int unsupported_caches(const char* what) {
  return fail(TQ_ERR_UNSUPPORTED,
              std::string(what) + ": supported channel groups are one group of d = 128 with 4 + 4 or 3 + 3 key / value "
                                  "bits, or two groups of d = 64 with (4 + 4, 3 + 3) or (3 + 3, 2 + 2) bits; caches and "
                                  "norms 16-byte aligned");
}

size_t tq_sparse_workspace_size(int B, int Hq, int Hkv, int D, int ngroups, int64_t max_len, int page_tokens,
                                int select) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || ngroups <= 0 || max_len < 0 || page_tokens <= 0 ||
      select < 1 || max_len > (int64_t)1 << 30 || (int64_t)select * page_tokens > (int64_t)1 << 30)
    return 0;
  return sparse_ws(B, Hq, Hkv, D, ngroups, page_tokens, (int)(max_len / page_tokens), select).total;
}

int tq_sparse_decode_attention(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                               const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                               const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len, float scale,
                               void* out, const tq_sparse_opts* opts, void* workspace, size_t ws_bytes,
                               tq_stream_t stream) {
  Range range_("tq_sparse_decode_attention");
  if (!opts) return fail(TQ_ERR_INVALID_ARG, "opts is NULL");
  const int page = opts->page_tokens;
  if (!opts->block_table || !opts->bounds) return fail(TQ_ERR_INVALID_ARG, "NULL block table or bounds");
  if (page <= 0 || page % 64 != 0 || max_len < 0 || max_len % page != 0)
    return fail(TQ_ERR_INVALID_ARG, "page_tokens must be a positive multiple of 64 that divides max_len");
  if (bad_dtype(opts->bounds_dtype) || opts->bounds_pages < 0) return fail(TQ_ERR_INVALID_ARG, "bad bounds");
  if (opts->select < 1 || opts->first < 0 || opts->last < 0)
    return fail(TQ_ERR_INVALID_ARG, "select must be at least 1, first and last not negative");
  if ((int64_t)opts->select * page > (int64_t)1 << 30) return fail(TQ_ERR_UNSUPPORTED, "select * page_tokens above 2^30");
  int r = check_decode_args(kctx, vctx, group_off, ngroups, q, q_dtype, kcache, vcache, seq_lens, B, Hq, Hkv, D,
                            max_len, out, page, true);
  if (r != TQ_OK) return r;
  if (B == 0) return TQ_OK;
  if ((r = check_cache_shape((int64_t)B * Hkv * ((Hq / Hkv + 3) / 4), (int64_t)B * Hq, max_len, "tq_sparse_decode_attention")) != TQ_OK) return r;
  if (!aligned(opts->bounds, 16) || !aligned(out, elem_size(q_dtype)) || !aligned(q, elem_size(q_dtype)))
    return fail(TQ_ERR_UNSUPPORTED, "bounds must be 16-byte aligned, q and out to their elements");
  if (!decode_caches_supported(kctx, vctx, ngroups, kcache, vcache)) return unsupported_caches("tq_sparse_decode_attention");
  const SparseWs W = sparse_ws(B, Hq, Hkv, D, ngroups, page, (int)(max_len / page), opts->select);
  if (!workspace || ws_bytes < W.total) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  if (!aligned(workspace, 16)) return fail(TQ_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  int64_t pool = INT64_MAX;
  for (int g = 0; g < ngroups; ++g) pool = std::min(pool, std::min(kcache[g].cap, vcache[g].cap));
  pool /= (int64_t)Hkv * page;
  if (pool * Hkv > INT32_MAX) return fail(TQ_ERR_UNSUPPORTED, "more than 2^31 - 1 (page, kv head) pairs");
  char* base = static_cast<char*>(workspace);
  DecodeView view;
  view.out_dtype = q_dtype;
  view.perm_Hq = Hq;
  view.perm_Hkv = Hkv;
  view.prepared = true;
  const int64_t sel_len = (int64_t)opts->select * page;
  const DecodeWs dw = decode_ws(B * Hkv, Hq / Hkv, 1, D, ngroups, sel_len);
  if (dw.nsplit > 512) return fail(TQ_ERR_UNSUPPORTED, "tq_sparse_decode_attention: more than 512 context splits");
  if ((r = launch_decode_prep(kctx, group_off, ngroups, opts->channel_perm, q, q_dtype, B * Hkv, Hq / Hkv, 1, D, sel_len,
                              base + W.decode, view, (cudaStream_t)stream)) != TQ_OK)
    return r;
  if ((r = launch_page_select(q, q_dtype, seq_lens, B, Hq, Hkv, D, max_len, pool, opts, workspace, W,
                              (cudaStream_t)stream)) != TQ_OK)
    return r;
  r = launch_decode_mma(kctx, vctx, group_off, ngroups, opts->channel_perm,
                        reinterpret_cast<const int32_t*>(base + W.vtable), page, q, q_dtype, kcache, vcache,
                        reinterpret_cast<const int32_t*>(base + W.vlen), B * Hkv, Hq / Hkv, 1, D,
                        sel_len, scale, out, base + W.decode, (cudaStream_t)stream, view);
  return r == kNotHandled ? fail(TQ_ERR_UNSUPPORTED, "tq_sparse_decode_attention: at most 512 context splits") : r;
}

size_t tq_tree_workspace_size(int B, int T, int Hq, int Hkv, int D, int ngroups, int64_t max_len) {
  if (B < 0 || T < 1 || T > 256 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D != 128 || ngroups <= 0 || max_len < 0 ||
      max_len > (int64_t)1 << 30)
    return 0;
  return tree_workspace_bytes(B, T, Hq, Hkv, max_len);
}

int tq_tree_attention(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                      const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                      const int32_t* seq_lens, const int32_t* draft_lens, const uint64_t* tree_mask, int B, int T,
                      int Hq, int Hkv, int D, int64_t max_len, float scale, void* out, const tq_decode_opts* opts,
                      void* workspace, size_t ws_bytes, tq_stream_t stream) {
  Range range_("tq_tree_attention");
  const int32_t* perm = opts ? opts->channel_perm : nullptr;
  const int32_t* table = opts ? opts->block_table : nullptr;
  const int page = table ? opts->page_tokens : 0;
  if (table && (page <= 0 || page % 64 != 0 || max_len % page != 0))
    return fail(TQ_ERR_INVALID_ARG, "page_tokens must be a positive multiple of 64 that divides max_len");
  if (T < 1 || T > 256) return fail(TQ_ERR_UNSUPPORTED, "T must be in [1, 256]");
  int r = check_decode_args(kctx, vctx, group_off, ngroups, q, q_dtype, kcache, vcache, seq_lens, B, Hq, Hkv, D,
                            max_len, out, page, true);
  if (r != TQ_OK) return r;
  if (B == 0) return TQ_OK;
  if ((r = check_cache_shape((int64_t)B * Hkv * ((Hq / Hkv + 3) / 4), (int64_t)B * T * Hq, max_len, "tq_tree_attention")) != TQ_OK) return r;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(perm, 16) || !aligned(tree_mask, 8))
    return fail(TQ_ERR_UNSUPPORTED, "q, out and the channel permutation must be 16-byte aligned, the mask 8-byte aligned");
  if (!decode_caches_supported(kctx, vctx, ngroups, kcache, vcache)) return unsupported_caches("tq_tree_attention");
  for (int g = 0; g < ngroups; ++g)
    if (kcache[g].cap > INT32_MAX || vcache[g].cap > INT32_MAX)
      return fail(TQ_ERR_UNSUPPORTED, "tq_tree_attention: a cache of more than 2^31 - 1 slots");
  const size_t need = tree_workspace_bytes(B, T, Hq, Hkv, max_len);
  if (!workspace || ws_bytes < need) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  if (!aligned(workspace, 16)) return fail(TQ_ERR_UNSUPPORTED, "workspace must be 16-byte aligned");
  return launch_tree_attention(kctx, vctx, group_off, ngroups, perm, table, page, q, q_dtype, kcache, vcache, seq_lens,
                               draft_lens, tree_mask, B, T, Hq, Hkv, D, max_len, scale, out, workspace,
                               (cudaStream_t)stream);
}

int tq_tree_mask(const int32_t* parent, int B, int T, uint64_t* mask) {
  if (!parent || !mask || B < 0 || T < 1 || T > 256) return fail(TQ_ERR_INVALID_ARG, "tq_tree_mask: bad arguments");
  const int W = (T + 63) / 64;
  for (int b = 0; b < B; ++b)
    for (int j = 0; j < T; ++j) {
      const int p = parent[(size_t)b * T + j];
      if (p < -1 || p >= j) return fail(TQ_ERR_INVALID_ARG, "tq_tree_mask: a parent must be in [-1, j)");
    }
  for (int b = 0; b < B; ++b)
    for (int j = 0; j < T; ++j) {
      const int p = parent[(size_t)b * T + j];
      uint64_t* row = mask + ((size_t)b * T + j) * W;
      for (int w = 0; w < W; ++w) row[w] = p >= 0 ? mask[((size_t)b * T + p) * W + w] : 0;
      row[j >> 6] |= 1ull << (j & 63);
    }
  return TQ_OK;
}

}  // extern "C"
