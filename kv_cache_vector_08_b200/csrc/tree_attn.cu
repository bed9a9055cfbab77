// Attention of a tree of drafted tokens over the packed cache, on the 5th-generation tensor cores.
//
// A sequence's cache holds its context and, in its last n tokens, the drafted ones.  Query row
// j (0 <= j < n) attends every context token and the drafted tokens i with bit i of mask[j]:
//   l_t = scale sum_g ||k_g|| ( <Pi q_g, c[idx]> + sqrt(pi/2)/d_g ||r_g|| <S q_g, 2 s - 1> )
//   out = sum_t softmax(l)_t v_t,   v_t[group g] = ||v_g|| Pi_vg^T c[idx]
// as in the decode kernels, for R = T rep query rows per kv head instead of rep.  With that many
// rows the contractions are worth decoding the cache into operands: for 128 rows and a tile of
// 64 tokens
//   S [128 x 64] = Q [128 x 256] K^T,   Q = (Pi q | sqrt(pi/2)/d S q),  K = ||k|| (c | +-||r||)
//   O [128 x 128] += P [128 x 64] V,    V = ||v|| c,   P = 2^(S - m)
// all operands fp16, sums fp32; the norms of the channel groups ride on the operands, so one
// product serves any grouping.
//
// CTA = 128 query rows of one (sequence, kv head) over one split of the tokens, two per SM; nine
// warps.  First the rows are projected (two products of the rows with Pi and S).  Then, tile by
// tile: warps 4-7 decode (thread = token x half of the head: code words come from global memory
// a tile ahead, byte-permute lookups make fp16 levels, K is written K-major, V with the channels
// contiguous as it lies in the cache); warp 8 issues the products; warps 0-3 (thread = row) turn
// S into P in place in tensor memory with a running maximum that moves only when it grew by 2^8,
// so that O, which stays in tensor memory, is seldom rescaled.  At the end O / l is rotated back
// by one more product, and written (one split) or left as a partial for the merge kernel.
//
// P carries a factor 2^7: between the 2^15 it can reach and the smallest fp16, weights down to
// 2^-31 of the row's largest count.
//
// Every wait is bounded; a timeout records an error code in the context's error word and the CTA
// winds down.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.cuh"
#include "mma_ops.cuh"
#include "sm100.cuh"

namespace tq {
namespace {

using namespace sm100;
using mmaops::prmt;

constexpr int kTD = 128;          // head dimension
constexpr int kTileTok = 64;      // tokens per tile: a tile never crosses a page
constexpr int kRows = 128;        // query rows per CTA
constexpr int kSoftWarps = 4, kDecWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kDecWarps + 1);
constexpr int kSoft = 32 * kSoftWarps, kDec = 32 * kDecWarps;
constexpr uint64_t kDrainNs = 2000000000ull;

// shared memory: the Q operand (first: rows and Pi for the projection), K and V operands
constexpr int kQBytes = kRows * 512, kKBytes = kTileTok * 512, kVBytes = kTileTok * 256;
constexpr int kOffK = kQBytes, kOffV = kOffK + kKBytes, kOffMisc = kOffV + kVBytes;
constexpr int kSmem = kOffMisc + 1024;
// tensor memory columns: S / P of even and odd tiles, O; the projections use all of them
constexpr int kTmemCols = 256, kColO = 128;

constexpr float kPShift = 7.f;    // P = 2^(l - m + 7)
constexpr float kGrow = 8.f;      // growth of the maximum (log2) that rescales O

struct TreeGroup {
  const uint8_t* kcodes;
  const uint16_t *knorm, *krnorm;
  const uint8_t* vcodes;
  const uint16_t* vnorm;
  uint32_t klo[2], khi[2];        // fp16 bytes of the signed level of each key code
  uint32_t vlo[2], vhi[2];        // fp16 bytes of the magnitudes of the value levels
  const __half *pi, *st, *piv;    // 16 Pi^T, 16 sqrt(pi/2)/d S^T of the keys, 16 Pi^T of the values ([d][d] fp16)
};

struct TreeArgs {
  TreeGroup g[2];
  int B, T, Hq, Hkv, rep, R, tiles_r, nsplit, chunk, words;
  int64_t max_len, npages;
  float scale_log2;               // |scale| log2(e)
  float sign;                     // sign of the scale
  const void* q;
  int q_dtype;
  void* out;
  const int32_t *seq_lens, *draft_lens;
  const uint64_t* mask;
  const int32_t *perm, *table;
  int page, max_pages;
  float* part;                    // [B Hkv R][nsplit][128] rotated partial results
  float2* ml;                     // [B Hkv R][nsplit] (maximum in log2, sum)
  uint64_t wait_ns;
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
// four consecutive elements (16- or 8-byte aligned)
__device__ __forceinline__ float4 load_any4(const void* p, int dtype, size_t i) {
  if (dtype == TQ_DTYPE_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == TQ_DTYPE_BF16)
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_any4(void* p, int dtype, size_t i, float4 v) {
  if (dtype == TQ_DTYPE_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
    return;
  }
  uint2 w;
  if (dtype == TQ_DTYPE_BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
}
__device__ __forceinline__ uint32_t h2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
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

// Operand of channels-contiguous rows (each row of 64 channels is 128 bytes, swizzled): the
// descriptor of a product that reads it with the channels as N and the rows as K.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block_bytes) {
  uint64_t d = desc_sw128(addr);
  d &= ~((uint64_t)0x3FFF << 16);
  return d | (uint64_t)(block_bytes >> 4) << 16;
}
constexpr uint32_t kMajorN = 1u << 16;     // instruction descriptor: B has N contiguous

// 16-byte chunk c of a 128-byte row, swizzled
__device__ __forceinline__ uint32_t swz(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

// A [rows][64 blocks] fp16 matrix of `cols` columns (a multiple of 64) into swizzled blocks of
// 64 columns, `rows` 128-byte rows each.
__device__ __forceinline__ void copy_matrix(uint8_t* dst, const __half* src, int rows, int cols, int t, int nt) {
  const int per = cols / 8;
  for (int e = t; e < rows * per; e += nt) {
    const int r = e / per, c = e - r * per;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + e);
    *reinterpret_cast<uint4*>(dst + (c >> 3) * rows * 128 + swz(r, c & 7)) = v;
  }
}

// The code words of one thread's 64 coordinates (two 32-coordinate groups of P words).
template <int P>
struct Words {
  uint32_t w[2 * P];
};
template <int P>
__device__ __forceinline__ void load_words(Words<P>& x, const uint8_t* rec) {
  if constexpr (P == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(rec) + i);
      x.w[2 * i] = v.x;
      x.w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(rec) + i);
      x.w[4 * i] = v.x; x.w[4 * i + 1] = v.y; x.w[4 * i + 2] = v.z; x.w[4 * i + 3] = v.w;
    }
  }
}
// Byte-permute selectors (low code bits) of slice u of group g, and its top bits at byte msbs.
template <int P>
__device__ __forceinline__ uint32_t low_sel(const Words<P>& x, int g, int u) {
  if constexpr (P == 4) return x.w[4 * g + u] & 0x77777777u;
  else if constexpr (P == 3) return (x.w[3 * g + (u & 1)] >> (2 * (u >> 1))) & 0x33333333u;
  else return (x.w[2 * g] >> u) & 0x11111111u;
}
template <int P>
__device__ __forceinline__ uint32_t top_bits(const Words<P>& x, int g, int u, int h) {
  if constexpr (P == 4) return h ? x.w[4 * g + u] << 4 : x.w[4 * g + u];
  else return x.w[P * g + P - 1] << (2 * u + h);
}

// Key rows: levels times the norm, and the residual signs times both norms.
template <int P>
__device__ __forceinline__ void decode_keys(const Words<P>& x, const TreeGroup& t, float n, float rn, uint8_t* lev,
                                            uint8_t* sgn, int row) {
  const uint32_t nn = h2_bits(n, n);
  const uint32_t rr = h2_bits(n * rn, n * rn) | 0x80008000u;    // (a set sign bit turns it positive)
  const int sw = row & 7;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t sel = low_sel<P>(x, g, u);
      uint32_t o[4], s[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sl = h ? sel >> 16 : sel;
        const uint32_t lb = prmt(t.klo[0], t.klo[1], sl), hb = prmt(t.khi[0], t.khi[1], sl);
        o[2 * h] = mul_h2(prmt(lb, hb, 0x5140u), nn);
        o[2 * h + 1] = mul_h2(prmt(lb, hb, 0x7362u), nn);
        const uint32_t tb = top_bits<P>(x, g, u, h);
        s[2 * h] = (prmt(tb, 0u, 0x1404u) & 0x80008000u) ^ rr;
        s[2 * h + 1] = (prmt(tb, 0u, 0x3424u) & 0x80008000u) ^ rr;
      }
      const int c = ((4 * g + u) ^ sw) << 4;
      *reinterpret_cast<uint4*>(lev + c) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(sgn + c) = make_uint4(s[0], s[1], s[2], s[3]);
    }
}
// Value rows: levels times the norm.
template <int P>
__device__ __forceinline__ void decode_values(const Words<P>& x, const TreeGroup& t, float n, uint8_t* dst, int row) {
  const uint32_t nn = h2_bits(n, n);
  const int sw = row & 7;
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t sel = low_sel<P>(x, g, u);
      uint32_t o[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sl = h ? sel >> 16 : sel;
        const uint32_t lb = prmt(t.vlo[0], t.vlo[1], sl);
        const uint32_t hb = prmt(t.vhi[0], t.vhi[1], sl) ^ (top_bits<P>(x, g, u, h) & 0x80808080u);
        o[2 * h] = mul_h2(prmt(lb, hb, 0x5140u), nn);
        o[2 * h + 1] = mul_h2(prmt(lb, hb, 0x7362u), nn);
      }
      *reinterpret_cast<uint4*>(dst + (((4 * g + u) ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

struct Bars {
  uint64_t proj, kfull, kempty, vfull, vempty, sfull[2], pfull[2], wfull, ofull, dfull, drain;
};

// The decoder warps of one half of the head: K of tile i + 1 before V of tile i, so that the
// next tile's logits are under way while this tile's weights are formed.
template <int PK, int PV, bool TWO>
__device__ __forceinline__ bool decode_loop(const TreeArgs& A, const TreeGroup& g, uint8_t* smem, Bars* bar, int half,
                                            int row, int b, int hk, int t0, int t1, int n, const volatile int* abort_v,
                                            int& code) {
  uint8_t* lev = smem + kOffK + half * (kTileTok * 128) + row * 128;
  uint8_t* sgn = lev + 2 * (kTileTok * 128);
  uint8_t* val = smem + kOffV + half * (kTileTok * 128) + row * 128;
  const int64_t slot0 = ((int64_t)b * A.Hkv + hk) * A.max_len;
  auto slot_of = [&](int i) -> int64_t {       // slot of this thread's token of tile i, or -1
    const int t = t0 + i * kTileTok + row;
    if (i >= n || t >= t1) return -1;
    if (!A.table) return slot0 + t;
    int pg = __ldg(A.table + (size_t)b * A.max_pages + t / A.page);
    if (pg < 0 || pg >= A.npages) {
      if (A.err) atomicCAS(A.err, 0, (int)kErrSlotRange);
      pg = 0;
    }
    return ((int64_t)pg * A.Hkv + hk) * A.page + t % A.page;
  };
  Words<PK> kw;
  Words<PV> vw;
  uint16_t kn = 0, kr = 0, vn = 0;
  // bytes of a record, and of this half's part of it
  constexpr int kRec = TWO ? PK * 8 : PK * 16, vRec = TWO ? PV * 8 : PV * 16;
  const int kOff = TWO ? 0 : half * PK * 8, vOff = TWO ? 0 : half * PV * 8;
  auto load_k = [&](int64_t s) {
    kn = kr = 0;
#pragma unroll
    for (int i = 0; i < 2 * PK; ++i) kw.w[i] = 0u;
    if (s >= 0) {
      load_words<PK>(kw, g.kcodes + s * kRec + kOff);
      kn = __ldg(g.knorm + s);
      kr = __ldg(g.krnorm + s);
    }
  };
  auto load_v = [&](int64_t s) {
    vn = 0;
#pragma unroll
    for (int i = 0; i < 2 * PV; ++i) vw.w[i] = 0u;
    if (s >= 0) {
      load_words<PV>(vw, g.vcodes + s * vRec + vOff);
      vn = __ldg(g.vnorm + s);
    }
  };
  auto f = [](uint16_t x) { return __half2float(__ushort_as_half(x)); };
  int64_t s1 = slot_of(0);
  load_k(s1);
  load_v(s1);
  for (int i = 0; i <= n; ++i) {
    const int64_t sv = s1;
    if (i < n) {
      s1 = slot_of(i + 1);
      if (!mbar_wait(&bar->kempty, (uint32_t)((i & 1) ^ 1), abort_v, A.wait_ns)) { code = 601; return false; }
      decode_keys<PK>(kw, g, f(kn), f(kr), lev, sgn, row);
      fence_proxy_async_smem();
      mbar_arrive(&bar->kfull);
      load_k(s1);
    }
    if (i > 0) {
      if (!mbar_wait(&bar->vempty, (uint32_t)(((i - 1) & 1) ^ 1), abort_v, A.wait_ns)) { code = 602; return false; }
      decode_values<PV>(vw, g, f(vn), val, row);
      fence_proxy_async_smem();
      mbar_arrive(&bar->vfull);
      if (i < n) load_v(sv);
    }
  }
  return true;
}

template <int PK0, int PV0, int PK1, int PV1, bool TWO>
__global__ void __launch_bounds__(kThreads, 2) tree_attn_kernel(const TreeArgs A) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + sizeof(Bars));
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* s_scale = reinterpret_cast<float*>(smem + kOffMisc + 512);      // [128] logit scale of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % A.nsplit;
  const int rt = (blockIdx.x / A.nsplit) % A.tiles_r;
  const int bh = blockIdx.x / (A.nsplit * A.tiles_r), b = bh / A.Hkv, hk = bh % A.Hkv;
  int len, nd;
  lens_of(A, b, len, nd);
  const int ctx = len - nd;
  const int r0 = rt * kRows;
  const int nrow = min(kRows, A.R - r0);                 // rows of this tile
  const int live = min(nrow, nd * A.rep - r0);           // those of drafted tokens that exist
  const int t0 = split * A.chunk, t1 = min(len, t0 + A.chunk);
  if (live <= 0 || t0 >= t1) {                           // nothing to attend: zeros (the merge writes its own)
    if (A.nsplit == 1)
      for (int e = threadIdx.x; e < nrow * kTD; e += kThreads)
        store_any(A.out, A.q_dtype, q_row(A, b, hk, r0 + e / kTD) * kTD + e % kTD, 0.f);
    return;
  }
  const int n = (t1 - t0 + kTileTok - 1) / kTileTok;
  if (threadIdx.x == 0) {
    mbar_init(&bar->proj, 1);
    mbar_init(&bar->kfull, kDec);
    mbar_init(&bar->kempty, 1);
    mbar_init(&bar->vfull, kDec);
    mbar_init(&bar->vempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->sfull[i], 1);
      mbar_init(&bar->pfull[i], kSoft);
    }
    mbar_init(&bar->wfull, kDec);
    mbar_init(&bar->ofull, kSoft);
    mbar_init(&bar->dfull, 1);
    mbar_init(&bar->drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kSoftWarps + kDecWarps) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // ------------------------------------------------------------------ projection of the rows
  // rows (fp16, scaled by a power of two so that the largest element is near 2^9) at 0, 16 Pi at
  // 32 KB, 16 kappa S in the K buffer
  copy_matrix(smem + 32768, A.g[0].pi, TWO ? 64 : 128, TWO ? 64 : 128, threadIdx.x, kThreads);
  copy_matrix(smem + kOffK, A.g[0].st, TWO ? 64 : 128, TWO ? 64 : 128, threadIdx.x, kThreads);
  if (TWO) {
    copy_matrix(smem + 32768 + 8192, A.g[1].pi, 64, 64, threadIdx.x, kThreads);
    copy_matrix(smem + kOffK + 8192, A.g[1].st, 64, 64, threadIdx.x, kThreads);
  }
  for (int r = warp; r < kRows; r += kThreads / 32) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < live) {
      const size_t base = q_row(A, b, hk, r0 + r) * kTD;
      if (A.perm) {
        const int4 ch = __ldg(reinterpret_cast<const int4*>(A.perm + (size_t)hk * kTD) + lane);
        auto get = [&](int c) {
          if (c >= 0 && c < kTD) return load_any(A.q, A.q_dtype, base + c);
          if (A.err) atomicCAS(A.err, 0, (int)kErrPermRange);
          return 0.f;
        };
        v = make_float4(get(ch.x), get(ch.y), get(ch.z), get(ch.w));
      } else {
        v = load_any4(A.q, A.q_dtype, base + 4 * lane);
      }
    }
    float mx = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int e = mx > 0.f && mx < INFINITY ? max(-110, min(110, 9 - ilogbf(mx))) : 0;
    const float up = ldexpf(A.sign, e);
    *reinterpret_cast<uint2*>(smem + (lane >> 4) * (kRows * 128) + swz(r, (lane >> 1) & 7) + 8 * (lane & 1)) =
        make_uint2(h2_bits(v.x * up, v.y * up), h2_bits(v.z * up, v.w * up));
    if (lane == 0) s_scale[r] = ldexpf(A.scale_log2, -e);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const volatile int* abort_v = abort_flag;
  auto fail = [&](int code) {
    atomicExch(abort_flag, 1);
    if (A.err) atomicCAS(A.err, 0, code);
  };
  auto wait = [&](uint64_t* x, uint32_t parity) { return mbar_wait(x, parity, abort_v, A.wait_ns); };
  // the same answer for the whole warp, which the tensor memory accesses behind it need
  auto wait_all = [&](uint64_t* x, uint32_t parity) { return __all_sync(0xffffffffu, wait(x, parity)) != 0; };
  bool ok = true;
  if (warp == kSoftWarps + kDecWarps && lane == 0) {
    // D columns 64 j: coordinates 64 j .. of Pi q, then (from 128 on) of kappa S q
    const uint32_t idesc = idesc_f16(kRows, 64, 0) | kMajorN;
    const uint32_t a0 = smem_u32(smem);
    for (int part = 0; part < 2; ++part)
      for (int j = 0; j < 2; ++j) {
        const uint32_t w = part ? smem_u32(smem + kOffK) : a0 + 32768;
        const uint32_t d = tmem + (uint32_t)(128 * part + 64 * j);
        for (int ks = 0; ks < (TWO ? 4 : 8); ++ks) {
          const uint32_t a = TWO ? a0 + j * (kRows * 128) + ks * 32 : a0 + (ks >> 2) * (kRows * 128) + (ks & 3) * 32;
          const uint32_t bb = w + j * (TWO ? 8192 : 16384) + ks * 2048;
          mma_ss(d, desc_sw128(a), desc_mn(bb, 8192), idesc, ks ? 1u : 0u);
        }
      }
    mma_commit(&bar->proj);
  }
  __syncwarp();
  if (!wait_all(&bar->proj, 0)) { fail(603); ok = false; }
  tc_fence_after();
  if (ok && warp < kSoftWarps + kDecWarps) {
    // warps 0-3: Pi q, warps 4-7: kappa S q; row = lane of the warp's quarter
    const int part = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t src = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + (uint32_t)(128 * part);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t v[32];
      tmem_ld32(src + 32 * c, v);
      tmem_ld_wait();
      uint8_t* dst = smem + (2 * part + (c >> 1)) * (kRows * 128);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = h2_bits(__uint_as_float(v[8 * k + 2 * i]) * (1.f / 16.f), __uint_as_float(v[8 * k + 2 * i + 1]) * (1.f / 16.f));
        *reinterpret_cast<uint4*>(dst + swz(r, 4 * (c & 1) + k)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  ok = *abort_v == 0;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax, thread = row
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    const bool warp_live = 32 * warp < live;
    const int j = (r0 + r) / A.rep;
    const bool row_live = r < live;
    const float sc = s_scale[r];
    // columns of the tile at ts that the row attends (tiles past the context or the split's end)
    auto kept = [&](int ts) -> uint64_t {
      const uint64_t keep = t1 - ts < 64 ? (1ull << (t1 - ts)) - 1 : ~0ull;
      const int d0 = ts - ctx;                       // drafted token of the tile's first column
      if (!row_live) return 0;
      if (d0 + 64 <= 0) return keep;
      if (!A.mask) return j < d0 ? 0 : j - d0 >= 63 ? keep : keep & ((2ull << (j - d0)) - 1);    // drafts up to j
      const uint64_t* mr = A.mask + ((size_t)b * A.T + j) * A.words;
      if (d0 < 0) return keep & ((__ldg(mr) << -d0) | ((1ull << -d0) - 1));
      const int w = d0 >> 6, sh = d0 & 63;
      uint64_t bits = w < A.words ? __ldg(mr + w) >> sh : 0;
      if (sh && w + 1 < A.words) bits |= __ldg(mr + w + 1) << (64 - sh);
      return keep & bits;
    };
    float m = -INFINITY, l = 0.f;
    for (int i = 0; ok && i < n; ++i) {
      if (!wait_all(&bar->sfull[i & 1], (uint32_t)((i >> 1) & 1))) { fail(604); ok = false; break; }
      tc_fence_after();
      if (warp_live) {
        const uint32_t col = lane_base + (uint32_t)(64 * (i & 1));
        const int ts = t0 + i * kTileTok;
        const bool whole = ts + kTileTok <= min(ctx, t1);
        const uint64_t keep = whole ? ~0ull : kept(ts);
        // S is read twice, 32 columns at a time: for the maximum, then for the weights (64 values
        // held at once would spill)
        float mt = -INFINITY;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t s[32];
          tmem_ld32(col + 32 * k, s);
          tmem_ld_wait();
          if (whole) {
#pragma unroll
            for (int c = 0; c < 32; ++c) mt = fmaxf(mt, __uint_as_float(s[c]));
          } else {
            const uint32_t kk = (uint32_t)(keep >> (32 * k));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if ((kk >> c) & 1) mt = fmaxf(mt, __uint_as_float(s[c]));
          }
        }
        mt = mt == -INFINITY ? mt : mt * sc;
        const bool first = m == -INFINITY;
        const bool grow = mt > m + kGrow;
        float f = 1.f;
        if (grow) {
          f = first ? 1.f : ex2(m - mt);
          m = mt;
          l *= f;
        }
        if (i > 0 && __any_sync(0xffffffffu, grow && !first)) {
          // O rows times f, once the products of the tile before are in
          if (!wait_all(&bar->vempty, (uint32_t)((i - 1) & 1))) { fail(605); ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(lane_base + kColO + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(lane_base + kColO + 16 * c, o);
          }
        }
        const float base = (m == -INFINITY ? 0.f : m) - kPShift;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t s[32], p[16];
          tmem_ld32(col + 32 * k, s);
          tmem_ld_wait();
          const uint32_t kk = (uint32_t)(keep >> (32 * k));
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float a = ex2(fmaf(__uint_as_float(s[2 * e]), sc, -base)), z = ex2(fmaf(__uint_as_float(s[2 * e + 1]), sc, -base));
            if (!whole) {
              a = (kk >> (2 * e)) & 1 ? a : 0.f;
              z = (kk >> (2 * e + 1)) & 1 ? z : 0.f;
            }
            l += a + z;
            p[e] = h2_bits(a, z);
          }
          tmem_st16(col + 16 * k, p);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      mbar_arrive(&bar->pfull[i & 1]);
    }
    if (ok && !wait_all(&bar->vempty, (uint32_t)((n - 1) & 1))) { fail(606); ok = false; }
    if (ok) {
      tc_fence_after();
      if (warp_live) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32], x[16];
          tmem_ld32(lane_base + kColO + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = h2_bits(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          tmem_st16(lane_base + 16 * c, x);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      mbar_arrive(&bar->ofull);
      if (!wait_all(&bar->dfull, 0)) { fail(607); ok = false; }
    }
    if (ok) {
      tc_fence_after();
      const size_t row = (size_t)bh * A.R + r0 + r;
      const size_t qr = r < nrow ? q_row(A, b, hk, r0 + r) * kTD : 0;
      if (warp_live) {
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[16];
          tmem_ld16(lane_base + kColO + 16 * c, o);
          tmem_ld_wait();
          const float inv16 = row_live ? 1.f / 16.f : 0.f;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            float4 v = make_float4(__uint_as_float(o[e]) * inv16, __uint_as_float(o[e + 1]) * inv16,
                                   __uint_as_float(o[e + 2]) * inv16, __uint_as_float(o[e + 3]) * inv16);
            if (!row_live) v = make_float4(0.f, 0.f, 0.f, 0.f);
            const int ch = 16 * c + e;
            if (r >= nrow) {
            } else if (A.nsplit > 1) {
              *reinterpret_cast<float4*>(A.part + (row * A.nsplit + split) * kTD + ch) = v;
            } else if (A.perm) {
              const int4 to = __ldg(reinterpret_cast<const int4*>(A.perm + (size_t)hk * kTD + ch));
              if (to.x >= 0 && to.x < kTD) store_any(A.out, A.q_dtype, qr + to.x, v.x);
              if (to.y >= 0 && to.y < kTD) store_any(A.out, A.q_dtype, qr + to.y, v.y);
              if (to.z >= 0 && to.z < kTD) store_any(A.out, A.q_dtype, qr + to.z, v.z);
              if (to.w >= 0 && to.w < kTD) store_any(A.out, A.q_dtype, qr + to.w, v.w);
            } else {
              store_any4(A.out, A.q_dtype, qr + ch, v);
            }
          }
        }
      } else if (r < nrow && A.nsplit == 1) {
        for (int e = 0; e < kTD; e += 4) store_any4(A.out, A.q_dtype, qr + e, make_float4(0.f, 0.f, 0.f, 0.f));
      }
      if (A.nsplit > 1 && r < nrow) A.ml[row * A.nsplit + split] = make_float2(m - kPShift, row_live ? l : 0.f);
    }
  } else if (warp < kSoftWarps + kDecWarps) {
    // ------------------------------------------------------------------ decoders
    const int dw = warp - kSoftWarps, half = dw >> 1, row = 32 * (dw & 1) + lane;
    int code = 0;
    if (ok) {
      if (half == 0) ok = decode_loop<PK0, PV0, TWO>(A, A.g[0], smem, bar, 0, row, b, hk, t0, t1, n, abort_v, code);
      else ok = decode_loop<PK1, PV1, TWO>(A, A.g[TWO ? 1 : 0], smem, bar, 1, row, b, hk, t0, t1, n, abort_v, code);
      if (!ok) fail(code);
    }
    // the value rotation into the K buffer, once the last logits are formed
    if (ok && !wait(&bar->kempty, (uint32_t)((n - 1) & 1))) { fail(608); ok = false; }
    if (ok) {
      const int t = threadIdx.x - kSoft;
      copy_matrix(smem + kOffK, A.g[0].piv, TWO ? 64 : 128, TWO ? 64 : 128, t, kDec);
      if (TWO) copy_matrix(smem + kOffK + 8192, A.g[1].piv, 64, 64, t, kDec);
      fence_proxy_async_smem();
      mbar_arrive(&bar->wfull);
    }
  } else if (lane == 0) {
    // ------------------------------------------------------------------ products
    const uint32_t qa = smem_u32(smem), ka = smem_u32(smem + kOffK), va = smem_u32(smem + kOffV);
    const uint32_t id_s = idesc_f16(kRows, kTileTok, 0), id_o = idesc_f16(kRows, kTD, 0) | kMajorN;
    for (int i = 0; ok && i <= n; ++i) {
      if (i < n) {
        if (!wait(&bar->kfull, (uint32_t)(i & 1))) { fail(609); ok = false; break; }
        // S(i) takes the columns of P(i - 2): its products are in
        if (i >= 2 && !wait(&bar->vempty, (uint32_t)(i & 1))) { fail(610); ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(64 * (i & 1));
        for (int k = 0; k < 16; ++k)
          mma_ss(d, desc_sw128(qa + (k >> 2) * (kRows * 128) + (k & 3) * 32),
                 desc_sw128(ka + (k >> 2) * (kTileTok * 128) + (k & 3) * 32), id_s, k ? 1u : 0u);
        mma_commit(&bar->sfull[i & 1]);
        mma_commit(&bar->kempty);
      }
      if (i > 0) {
        const int p = i - 1;
        if (!wait(&bar->pfull[p & 1], (uint32_t)((p >> 1) & 1)) || !wait(&bar->vfull, (uint32_t)(p & 1))) {
          fail(611);
          ok = false;
          break;
        }
        tc_fence_after();
        for (int k = 0; k < 4; ++k)
          mma_ts(tmem + kColO, tmem + (uint32_t)(64 * (p & 1) + 8 * k), desc_mn(va + k * 2048, kTileTok * 128), id_o,
                 p > 0 || k > 0 ? 1u : 0u);
        mma_commit(&bar->vempty);
      }
    }
    if (ok && (!wait(&bar->wfull, 0) || !wait(&bar->ofull, 0))) { fail(612); ok = false; }
    if (ok) {
      // out = O / l times Pi of the values
      tc_fence_after();
      if (TWO) {
        const uint32_t id = idesc_f16(kRows, 64, 0);
        for (int g = 0; g < 2; ++g)
          for (int k = 0; k < 4; ++k)
            mma_ts(tmem + kColO + 64 * g, tmem + (uint32_t)(32 * g + 8 * k), desc_sw128(ka + g * 8192 + k * 32), id, k ? 1u : 0u);
      } else {
        const uint32_t id = idesc_f16(kRows, kTD, 0);
        for (int k = 0; k < 8; ++k)
          mma_ts(tmem + kColO, tmem + (uint32_t)(8 * k), desc_sw128(ka + (k >> 2) * (kTD * 128) + (k & 3) * 32), id, k ? 1u : 0u);
      }
      mma_commit(&bar->dfull);
    }
    mma_commit(&bar->drain);
    mbar_wait(&bar->drain, 0, nullptr, kDrainNs);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kDecWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Log-sum-exp merge of the splits, one warp per row, lane = 4 channels.
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs A) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)A.B * A.Hkv * A.R) return;
  const int lane = threadIdx.x & 31;
  const int r = (int)(row % A.R), bh = (int)(row / A.R), b = bh / A.Hkv, hk = bh % A.Hkv;
  int len, nd;
  lens_of(A, b, len, nd);
  const int ns = r / A.rep < nd ? (len + A.chunk - 1) / A.chunk : 0;     // splits that hold tokens
  const float2* ml = A.ml + row * A.nsplit;
  const float4* part = reinterpret_cast<const float4*>(A.part + row * A.nsplit * kTD) + lane;
  float m = -INFINITY;
  for (int s = lane; s < ns; s += 32)
    if (ml[s].y != 0.f) m = fmaxf(m, ml[s].x);       // (a split that attends nothing has no maximum)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float L = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < ns; ++s) {
    const float2 x = ml[s];
    const float4 v = part[s * (kTD / 4)];
    if (x.y == 0.f) continue;
    const float w = ex2(x.x - m) * x.y;
    L += w;
    a.x = fmaf(w, v.x, a.x);
    a.y = fmaf(w, v.y, a.y);
    a.z = fmaf(w, v.z, a.z);
    a.w = fmaf(w, v.w, a.w);
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
  const size_t base = q_row(A, b, hk, r) * kTD;
  if (A.perm) {
    const int4 to = __ldg(reinterpret_cast<const int4*>(A.perm + (size_t)hk * kTD) + lane);
    if (to.x >= 0 && to.x < kTD) store_any(A.out, A.q_dtype, base + to.x, a.x);
    if (to.y >= 0 && to.y < kTD) store_any(A.out, A.q_dtype, base + to.y, a.y);
    if (to.z >= 0 && to.z < kTD) store_any(A.out, A.q_dtype, base + to.z, a.z);
    if (to.w >= 0 && to.w < kTD) store_any(A.out, A.q_dtype, base + to.w, a.w);
  } else {
    store_any4(A.out, A.q_dtype, base + 4 * lane, a);
  }
}

struct TreeWs {
  size_t part, ml, total;
  int nsplit, chunk;
};

// Splits of the tokens: as many as give the shortest modelled time, waves of CTAs (two per SM)
// times (tiles per CTA + the cost of a CTA's start and end, about kEdge tiles).
constexpr int kEdge = 8, kMaxSplit = 128;

TreeWs tree_ws(int B, int T, int Hq, int Hkv, int64_t max_len) {
  TreeWs w{};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
    cudaGetLastError();
    sms = 148;
  }
  const int R = T * (Hq / Hkv);
  const int64_t rows = (int64_t)B * Hkv * R, ctas = (int64_t)B * Hkv * ((R + kRows - 1) / kRows);
  const int64_t tiles = std::max<int64_t>(1, (max_len + kTileTok - 1) / kTileTok);
  int64_t best = 1;
  double best_t = 1e300;
  for (int64_t s = 1; s <= std::min<int64_t>(kMaxSplit, tiles); ++s) {
    const int64_t per = (tiles + s - 1) / s;
    if (s > 1 && (tiles + per - 1) / per < s) continue;        // same split as a smaller s
    const double t = (double)((std::max<int64_t>(1, ctas) * s + 2 * sms - 1) / (2 * sms)) * (double)(per + kEdge);
    if (t < best_t - 1e-9) {
      best_t = t;
      best = s;
    }
  }
  const int64_t per = (tiles + best - 1) / best;
  w.chunk = (int)(per * kTileTok);
  w.nsplit = (int)((tiles + per - 1) / per);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.ml = w.nsplit > 1 ? up((size_t)rows * w.nsplit * kTD * sizeof(float)) : 0;
  w.total = w.nsplit > 1 ? w.ml + up((size_t)rows * w.nsplit * sizeof(float2)) : 256;
  return w;
}

template <int PK0, int PV0, int PK1, int PV1, bool TWO>
int launch_main(const TreeArgs& A, unsigned ctas, cudaStream_t st) {
  cudaError_t e = ensure_smem_attrs<tree_attn_kernel<PK0, PV0, PK1, PV1, TWO>>(kSmem, true);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tree_attn_kernel)");
  tree_attn_kernel<PK0, PV0, PK1, PV1, TWO><<<ctas, kThreads, kSmem, st>>>(A);
  count_launch();
  return check_launch("tree_attn_kernel");
}

uint32_t half_bits(float v) {
  const __half h = __float2half_rn(v);
  return *reinterpret_cast<const uint16_t*>(&h);
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
  A.B = B; A.T = T; A.Hq = Hq; A.Hkv = Hkv; A.rep = Hq / Hkv; A.R = T * A.rep;
  A.tiles_r = (A.R + kRows - 1) / kRows;
  A.nsplit = W.nsplit; A.chunk = W.chunk;
  A.words = (T + 63) / 64;
  A.max_len = max_len;
  A.scale_log2 = fabsf(scale) * 1.4426950408889634f;
  A.sign = scale < 0.f ? -1.f : 1.f;
  A.q = q; A.q_dtype = q_dtype; A.out = out;
  A.seq_lens = seq_lens; A.draft_lens = draft_lens; A.mask = mask; A.perm = perm; A.table = table;
  A.part = reinterpret_cast<float*>(ws);
  A.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + W.ml);
  A.wait_ns = pipeline_wait_ns();
  A.err = kctx[0]->dev_err;
  int64_t pool = INT64_MAX;
  for (int g = 0; g < G; ++g) {
    TreeGroup& t = A.g[g];
    t.kcodes = kc[g].codes; t.knorm = kc[g].norm; t.krnorm = kc[g].rnorm; t.vcodes = vc[g].codes; t.vnorm = vc[g].norm;
    const Codebook &kb = kctx[g]->cb, &vb = vctx[g]->cb;
    for (int i = 0; i < kb.K && i < 8; ++i) {
      t.klo[i / 4] |= (half_bits(kb.cc[i]) & 0xFF) << (8 * (i % 4));
      t.khi[i / 4] |= (half_bits(kb.cc[i]) >> 8) << (8 * (i % 4));
    }
    for (int i = 0; i < vb.K / 2 && i < 8; ++i) {
      t.vlo[i / 4] |= (half_bits(vb.c[vb.K / 2 + i]) & 0xFF) << (8 * (i % 4));
      t.vhi[i / 4] |= (half_bits(vb.c[vb.K / 2 + i]) >> 8) << (8 * (i % 4));
    }
    t.pi = static_cast<const __half*>(kctx[g]->PiT_f16);
    t.st = static_cast<const __half*>(kctx[g]->ST_f16);
    t.piv = static_cast<const __half*>(vctx[g]->PiT_f16);
    pool = std::min(pool, std::min(kc[g].cap, vc[g].cap));
  }
  if (table) {
    A.page = page;
    A.max_pages = (int)(max_len / page);
    A.npages = pool / ((int64_t)Hkv * page);
  }
  const unsigned ctas = (unsigned)((int64_t)B * Hkv * A.tiles_r * A.nsplit);
  int r;
  if (G == 1 && kctx[0]->lay.planes == 4) r = launch_main<4, 4, 4, 4, false>(A, ctas, st);
  else if (G == 1) r = launch_main<3, 3, 3, 3, false>(A, ctas, st);
  else if (kctx[0]->lay.planes == 4) r = launch_main<4, 4, 3, 3, true>(A, ctas, st);
  else r = launch_main<3, 3, 2, 2, true>(A, ctas, st);
  if (r != TQ_OK || A.nsplit == 1) return r;
  tree_merge_kernel<<<(unsigned)(((int64_t)B * Hkv * A.R + 7) / 8), 256, 0, st>>>(A);
  count_launch();
  return check_launch("tree_merge_kernel");
}

}  // namespace tq
