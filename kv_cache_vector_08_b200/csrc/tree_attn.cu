// Attention of a tree of drafted tokens over the packed cache.
//
// A sequence's cache holds its context and, in its last n tokens, the drafted ones.  Query row
// j (0 <= j < n) attends every context token and the drafted tokens i with bit i of mask[j]:
//   l_t = scale sum_g ||k_g|| ( <Pi q_g, c[idx]> + sqrt(pi/2)/d_g ||r_g|| <S q_g, 2 s - 1> )
//   out = sum_t softmax(l)_t v_t,   v_t[group g] = ||v_g|| Pi_vg^T c[idx]
// as in the decode kernels, for T rep query rows per kv head instead of rep.
//
// Three kernels: the rows' projections, partial softmax states over splits of the context,
// and their merge with the inverse value rotation.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.cuh"

namespace tq {
namespace {

constexpr int kTD = 128;        // head dimension
constexpr int kTileTok = 64;    // tokens per tile: a tile never crosses a page
constexpr int kRowsCta = 8;

struct TreeGroup {
  const uint8_t* kcodes;
  const uint16_t *knorm, *krnorm;
  const uint8_t* vcodes;
  const uint16_t* vnorm;
  float kcc[8], vcc[16];        // level of each code
  int off, dg, pk, pv;
  const float *pit, *st, *piv;  // Pi^T, S^T of the keys, Pi of the values
  float coef;
};

struct TreeArgs {
  TreeGroup g[2];
  int G, B, T, Hq, Hkv, rep, nsplit, chunk, words;
  int64_t max_len, npages;
  float scale;
  const void* q;
  int q_dtype;
  void* out;
  const int32_t *seq_lens, *draft_lens;
  const uint64_t* mask;
  const int32_t *perm, *table;
  int page, max_pages;
  float* qp;                    // [B][Hkv][T rep][2][128]
  float* part;                  // [B][Hkv][T rep][nsplit][130]
  int* err;
};

__device__ __forceinline__ float load_any(const void* p, int dtype, size_t i) {
  if (dtype == TQ_DTYPE_F32) return static_cast<const float*>(p)[i];
  if (dtype == TQ_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void store_any(void* p, int dtype, size_t i, float v) {
  if (dtype == TQ_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == TQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Tokens of sequence b and the drafted ones among them.
__device__ __forceinline__ void lens_of(const TreeArgs& A, int b, int& len, int& nd) {
  len = (int)max((int64_t)0, min((int64_t)A.seq_lens[b], A.max_len));
  nd = min(len, A.T);
  if (A.draft_lens) nd = max(0, min(nd, A.draft_lens[b]));
}

// Row r of (b, hk) is query head hk rep + r % rep of drafted token r / rep.
__device__ __forceinline__ size_t q_row(const TreeArgs& A, int b, int hk, int r) {
  return ((size_t)b * A.T + r / A.rep) * A.Hq + hk * A.rep + r % A.rep;
}

__global__ void __launch_bounds__(kTD) tree_prep_kernel(const TreeArgs A) {
  __shared__ float xs[kTD];
  const int R = A.T * A.rep;
  const int64_t row = blockIdx.x;
  const int r = (int)(row % R), bh = (int)(row / R), b = bh / A.Hkv, hk = bh % A.Hkv;
  const int c = threadIdx.x;
  int ch = A.perm ? A.perm[(size_t)hk * kTD + c] : c;
  const bool ok = ch >= 0 && ch < kTD;
  if (!ok && A.err) atomicCAS(A.err, 0, (int)kErrPermRange);
  xs[c] = ok ? load_any(A.q, A.q_dtype, q_row(A, b, hk, r) * kTD + ch) : 0.f;
  __syncthreads();
  const bool second = A.G > 1 && c >= A.g[1].off;
  const TreeGroup& g = A.g[second ? 1 : 0];
  const int o = c - g.off;
  float a = 0.f, s = 0.f;
  for (int j = 0; j < g.dg; ++j) {
    a = fmaf(g.pit[(size_t)j * g.dg + o], xs[g.off + j], a);
    s = fmaf(g.st[(size_t)j * g.dg + o], xs[g.off + j], s);
  }
  A.qp[(size_t)row * 2 * kTD + c] = a;
  A.qp[(size_t)row * 2 * kTD + kTD + c] = s * g.coef;
}

__global__ void __launch_bounds__(256) tree_simple_kernel(const TreeArgs A) {
  extern __shared__ float sm[];
  float* kt = sm;                               // [64][129] levels times norm, then the values
  float* ks = kt + kTileTok * (kTD + 1);        // [64][129] signs times both norms
  float* qs = ks + kTileTok * (kTD + 1);        // [8][256]
  float* ps = qs + kRowsCta * 2 * kTD;          // [8][64]
  const int R = A.T * A.rep, nrb = (R + kRowsCta - 1) / kRowsCta;
  const int bh = blockIdx.y / nrb, rb = blockIdx.y % nrb, b = bh / A.Hkv, hk = bh % A.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int len, nd;
  lens_of(A, b, len, nd);
  const int ctx = len - nd;
  const int r = rb * kRowsCta + warp, j = r / A.rep;
  const bool live = r < R && j < nd;
  const int t0 = blockIdx.x * A.chunk, t1 = min(len, t0 + A.chunk);
  for (int e = threadIdx.x; e < kRowsCta * 2 * kTD; e += 256) {
    const int rr = rb * kRowsCta + e / (2 * kTD);
    qs[e] = rr < R ? A.qp[((size_t)bh * R + rr) * 2 * kTD + e % (2 * kTD)] : 0.f;
  }
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int ts = t0; ts < t1; ts += kTileTok) {
    int64_t slot;
    if (A.table) {
      int pg = A.table[(size_t)b * A.max_pages + ts / A.page];
      if (pg < 0 || pg >= A.npages) {
        if (A.err) atomicCAS(A.err, 0, (int)kErrSlotRange);
        pg = 0;
      }
      slot = ((int64_t)pg * A.Hkv + hk) * A.page + ts % A.page;
    } else {
      slot = (int64_t)bh * A.max_len + ts;
    }
    auto fill = [&](bool keys) {
      for (int e = threadIdx.x; e < kTileTok * 4; e += 256) {
        const int t = e >> 2, gr = e & 3;
        const TreeGroup& g = A.g[A.G > 1 && gr >= 2 ? 1 : 0];
        const int P = keys ? g.pk : g.pv, lg = gr - g.off / 32;
        const bool in = ts + t < t1;
        const int64_t s = slot + (in ? t : 0);
        uint32_t w[4];
        const uint32_t* rec = reinterpret_cast<const uint32_t*>((keys ? g.kcodes : g.vcodes) + s * (P * g.dg / 8)) + lg * P;
        for (int i = 0; i < P; ++i) w[i] = rec[i];
        const float n = in ? __half2float(__ushort_as_half((keys ? g.knorm : g.vnorm)[s])) : 0.f;
        const float rn = keys && in ? n * __half2float(__ushort_as_half(g.krnorm[s])) : 0.f;
        for (int i = 0; i < 32; ++i) {
          const uint32_t code = group_code(w, P, i);
          if (keys) {
            kt[t * (kTD + 1) + gr * 32 + i] = n * g.kcc[code & ((1u << (P - 1)) - 1u)];
            ks[t * (kTD + 1) + gr * 32 + i] = (code >> (P - 1)) & 1u ? rn : -rn;
          } else {
            kt[t * (kTD + 1) + gr * 32 + i] = n * g.vcc[code];
          }
        }
      }
    };
    __syncthreads();
    fill(true);
    __syncthreads();
    float lg[2];
    for (int u = 0; u < 2; ++u) {
      const int t = lane + 32 * u, tok = ts + t;
      float a = 0.f;
      for (int c = 0; c < kTD; ++c) {
        a = fmaf(qs[warp * 2 * kTD + c], kt[t * (kTD + 1) + c], a);
        a = fmaf(qs[warp * 2 * kTD + kTD + c], ks[t * (kTD + 1) + c], a);
      }
      bool keep = live && tok < t1;
      if (keep && tok >= ctx) {
        const int i = tok - ctx;
        keep = A.mask ? (A.mask[((size_t)b * A.T + j) * A.words + (i >> 6)] >> (i & 63)) & 1 : i <= j;
      }
      lg[u] = keep ? a * A.scale : -INFINITY;
    }
    float mt = fmaxf(lg[0], lg[1]);
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const float mn = fmaxf(m, mt);
    if (mn > m) {
      const float f = __expf(m - mn);
      l *= f;
      for (int c = 0; c < 4; ++c) acc[c] *= f;
      m = mn;
    }
    for (int u = 0; u < 2; ++u) {
      const float p = lg[u] == -INFINITY ? 0.f : __expf(lg[u] - m);
      l += p;
      ps[warp * kTileTok + lane + 32 * u] = p;
    }
    __syncthreads();
    fill(false);
    __syncthreads();
    for (int t = 0; t < kTileTok; ++t) {
      const float p = ps[warp * kTileTok + t];
      for (int c = 0; c < 4; ++c) acc[c] = fmaf(p, kt[t * (kTD + 1) + lane + 32 * c], acc[c]);
    }
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (r >= R) return;
  float* dst = A.part + (((size_t)bh * R + r) * A.nsplit + blockIdx.x) * (kTD + 2);
  if (lane == 0) { dst[0] = m; dst[1] = l; }
  for (int c = 0; c < 4; ++c) dst[2 + lane + 32 * c] = acc[c];
}

__global__ void __launch_bounds__(kTD) tree_merge_kernel(const TreeArgs A) {
  __shared__ float v[kTD];
  const int R = A.T * A.rep;
  const int64_t row = blockIdx.x;
  const int r = (int)(row % R), bh = (int)(row / R), b = bh / A.Hkv, hk = bh % A.Hkv;
  const int c = threadIdx.x;
  const float* p = A.part + (size_t)row * A.nsplit * (kTD + 2);
  float m = -INFINITY;
  for (int s = 0; s < A.nsplit; ++s) m = fmaxf(m, p[s * (kTD + 2)]);
  float l = 0.f, a = 0.f;
  for (int s = 0; s < A.nsplit; ++s) {
    const float ms = p[s * (kTD + 2)], f = ms == -INFINITY ? 0.f : __expf(ms - m);
    l = fmaf(f, p[s * (kTD + 2) + 1], l);
    a = fmaf(f, p[s * (kTD + 2) + 2 + c], a);
  }
  v[c] = l > 0.f ? a / l : 0.f;
  __syncthreads();
  const bool second = A.G > 1 && c >= A.g[1].off;
  const TreeGroup& g = A.g[second ? 1 : 0];
  const int o = c - g.off;
  float x = 0.f;
  for (int i = 0; i < g.dg; ++i) x = fmaf(g.piv[(size_t)i * g.dg + o], v[g.off + i], x);
  const int ch = A.perm ? A.perm[(size_t)hk * kTD + c] : c;
  if (ch >= 0 && ch < kTD) store_any(A.out, A.q_dtype, q_row(A, b, hk, r) * kTD + ch, x);
}

struct TreeWs {
  size_t qp, part, total;
  int nsplit, chunk;
};

TreeWs tree_ws(int B, int T, int Hq, int Hkv, int64_t max_len) {
  TreeWs w{};
  const int64_t rows = (int64_t)B * T * Hq;
  const int64_t ctas = (int64_t)B * Hkv * ((T * (Hq / Hkv) + kRowsCta - 1) / kRowsCta);
  const int64_t tiles = std::max<int64_t>(1, (max_len + kTileTok - 1) / kTileTok);
  const int64_t want = std::min<int64_t>(std::min<int64_t>(tiles, 64), std::max<int64_t>(1, 592 / std::max<int64_t>(1, ctas)));
  const int64_t per = (tiles + want - 1) / want;
  w.chunk = (int)(per * kTileTok);
  w.nsplit = (int)((tiles + per - 1) / per);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.part = up((size_t)rows * 2 * kTD * sizeof(float));
  w.total = w.part + up((size_t)rows * w.nsplit * (kTD + 2) * sizeof(float));
  return w;
}

}  // namespace

size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int64_t max_len) {
  return tree_ws(B, T, Hq, Hkv, max_len).total;
}

int launch_tree_attention(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* off, int G,
                          const int32_t* perm, const int32_t* table, int page, const void* q, int q_dtype,
                          const tq_packed* kc, const tq_packed* vc, const int32_t* seq_lens,
                          const int32_t* draft_lens, const uint64_t* mask, int B, int T, int Hq, int Hkv, int D,
                          int64_t max_len, float scale, void* out, void* ws, cudaStream_t st) {
  const TreeWs W = tree_ws(B, T, Hq, Hkv, max_len);
  TreeArgs A{};
  A.G = G; A.B = B; A.T = T; A.Hq = Hq; A.Hkv = Hkv; A.rep = Hq / Hkv; A.nsplit = W.nsplit; A.chunk = W.chunk;
  A.words = (T + 63) / 64;
  A.max_len = max_len; A.scale = scale; A.q = q; A.q_dtype = q_dtype; A.out = out;
  A.seq_lens = seq_lens; A.draft_lens = draft_lens; A.mask = mask; A.perm = perm; A.table = table;
  A.qp = reinterpret_cast<float*>(static_cast<char*>(ws) + W.qp);
  A.part = reinterpret_cast<float*>(static_cast<char*>(ws) + W.part);
  A.err = kctx[0]->dev_err;
  int64_t pool = INT64_MAX;
  for (int g = 0; g < G; ++g) {
    TreeGroup& t = A.g[g];
    t.kcodes = kc[g].codes; t.knorm = kc[g].norm; t.krnorm = kc[g].rnorm; t.vcodes = vc[g].codes; t.vnorm = vc[g].norm;
    for (int i = 0; i < 8; ++i) t.kcc[i] = i < kctx[g]->cb.K ? kctx[g]->cb.cc[i] : 0.f;
    for (int i = 0; i < 16; ++i) t.vcc[i] = i < vctx[g]->cb.K ? vctx[g]->cb.cc[i] : 0.f;
    t.off = off[g]; t.dg = kctx[g]->lay.d; t.pk = kctx[g]->lay.planes; t.pv = vctx[g]->lay.planes;
    t.pit = kctx[g]->PiT; t.st = kctx[g]->ST; t.piv = vctx[g]->Pi;
    t.coef = kctx[g]->sqrt_pi_over_2_over_m;
    pool = std::min(pool, std::min(kc[g].cap, vc[g].cap));
  }
  if (table) {
    A.page = page;
    A.max_pages = (int)(max_len / page);
    A.npages = pool / ((int64_t)Hkv * page);
  }
  const int R = T * A.rep, nrb = (R + kRowsCta - 1) / kRowsCta;
  tree_prep_kernel<<<(unsigned)((int64_t)B * Hkv * R), kTD, 0, st>>>(A);
  count_launch();
  int r = check_launch("tree_prep_kernel");
  if (r != TQ_OK) return r;
  const int dyn = (2 * kTileTok * (kTD + 1) + kRowsCta * 2 * kTD + kRowsCta * kTileTok) * (int)sizeof(float);
  cudaError_t e = ensure_smem_attrs<tree_simple_kernel>(dyn, false);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tree_simple_kernel)");
  tree_simple_kernel<<<dim3(W.nsplit, (unsigned)(B * Hkv * nrb)), 256, dyn, st>>>(A);
  count_launch();
  if ((r = check_launch("tree_simple_kernel")) != TQ_OK) return r;
  tree_merge_kernel<<<(unsigned)((int64_t)B * Hkv * R), kTD, 0, st>>>(A);
  count_launch();
  return check_launch("tree_merge_kernel");
}

}  // namespace tq
