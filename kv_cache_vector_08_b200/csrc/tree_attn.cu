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
// CTA = up to 128 query rows of one (sequence, kv head) over one split of the tokens, one per SM.
// First the rows are projected (two products of the rows with Pi and S); Q then stays in tensor
// memory as the A operand, because a product that fetches both operands from shared memory is
// bound by that at 64 columns (measured: 768 cycles of a tile's S instead of 256).  Then a pipeline
// of tiles, four deep in K, V and S:
//   decoders (12 warps, three sets that take every third tile; thread = token x half of the head): code
//     words come from global memory a tile ahead, byte-permute lookups make fp16 levels; K is
//     written K-major, V with the channels contiguous, as it lies in the cache;
//   products (one warp): S of tile i, then O += P V of tile i - 2;
//   softmax (4 warps, thread = row): S to P in place in tensor memory, with a running maximum
//     that moves only when it grew by 2^12, so that O, which stays in tensor memory, is seldom
//     rescaled.
// Rows that fill a half or a quarter of the 128 lanes are repeated in the others (fold 2 or 4), and
// each copy takes its half or quarter of the tile's columns, with zeros in the rest of its P.  The
// products cost the same, the exponentials spread over all lanes.  The copies' sums meet at the end.
// At last O / l, each row scaled by a power of two of its own as the queries are, is rotated back by
// one more product, and written (one split) or left as a partial for the merge kernel.
//
// The levels of a codebook enter scaled by a factor for which fp16 holds them almost exactly
// (tq_init looks for it); the projection and the last product take the factor out.
//
// Roundings: every operand is fp16 (2^-11), whatever the queries' type; sums, logits, maxima and sums of
// the softmax are 32-bit.  What each operand costs, alone, of a row's size in a model of the arithmetic (3
// bits, 4,096 tokens, normal queries at scale 1 / sqrt(128)): keys 6.3e-4 (level times norm, and one product of both
// norms a token), the high halves of Pi and S 4.0e-4, projected queries 3.8e-4, rows before the rotation
// back 2.1e-4, that rotation's high half 2.1e-4, values 1.8e-4, weights 0.6e-4, query rows 0 from 16 bits;
// together 9.3e-4.  They are kept because the large ones are the tile's own operands: low halves of keys
// and queries would make S three products, 1,536 cycles a tile where it has 512 (and the tile 1,370),
// while low halves of the matrices and the output alone would leave 8.6e-4.  A bf16 result is rounded by
// 1.7e-3 of its size in any case.
//
// P carries a factor 2^3: between the 2^15 it can reach (2^12 before the maximum moves) and the smallest
// fp16, weights down to 2^-27 of the row's largest count at least.
//
// Bound: of the about 1,370 cycles of a tile at 64 rows, the products need 768 (the same for any row count
// up to 128), the shared memory 768 (K and V written once, read once by the products), the issue slots 810
// and the integer pipe of decoders and softmax 690; each waits on the others.  Products alone took 1,030
// cycles a tile, decoders alone 1,160.  64 sequences of up to 8,192 tokens, 16 drafts, 8 kv heads of 4
// query heads: 362 us (134 GFLOP, 412 MB; the first kernel of this shape, with one tile in flight, 723 us).
// One sequence of 131,072 tokens, 63 drafts: 248 us, 203 GFLOP, 0.82 PFLOP/s.
// Tried: two warps for the products, S and P V (391 us, spills); two softmax groups of two S buffers each
// (404 us); four decoder sets (no change).
//
// Every wait is bounded; a timeout records an error code in the context's error word and the CTA
// winds down.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "elem.cuh"
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
constexpr int kSoftWarps = 4, kDecWarps = 12, kMmaWarp = kSoftWarps + kDecWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr int kDecSet = 4, kSets = kDecWarps / kDecSet;   // warps that decode one tile, sets of them
constexpr int kStages = 4;                  // tiles in flight (K, V, S)
constexpr int kAhead = 2;                   // S runs this many tiles ahead of O += P V
constexpr uint64_t kDrainNs = 2000000000ull;

// shared memory: K and V stages (first: the rows, 16 Pi and 16 kappa S of the projection; at the end:
// Pi of the values and the copies' results)
constexpr int kKBytes = kTileTok * 512, kVBytes = kTileTok * 256;
constexpr int kOffV = kStages * kKBytes, kOffMisc = kOffV + kStages * kVBytes;
constexpr int kSmem = kOffMisc + 2048;
constexpr int kOffPi = 32768, kOffS = 65536;             // of the projection
constexpr int kOffSum = 32768;                           // copies' results, rows of kSumLd floats
constexpr int kSumLd = 132;
// tensor memory columns: Q, O, four S / P buffers (the projections use the latter)
constexpr int kTmemCols = 512, kColQ = 0, kColO = 128, kColS = 256;

constexpr float kPShift = 3.f;    // P = 2^(l - m + 3)
constexpr float kGrow = 12.f;     // growth of the maximum (log2) that rescales O

struct TreeGroup {
  const uint8_t* kcodes;
  const uint16_t *knorm, *krnorm;
  const uint8_t* vcodes;
  const uint16_t* vnorm;
  uint32_t klo[2], khi[2];        // fp16 bytes of the signed level of each key code
  uint32_t vlo[2], vhi[2];        // fp16 bytes of the magnitudes of the value levels
  float kinv, vinv;               // 1 / (16 factor) of the key and value levels
  const __half *pi, *st, *piv;    // 16 Pi^T, 16 sqrt(pi/2)/d S^T of the keys, 16 Pi^T of the values ([d][d] fp16)
};

struct TreeArgs {
  TreeGroup g[2];
  int B, T, Hq, Hkv, rep, R, fold, tiles_r, nsplit, chunk, words;
  int sort;                       // sequences in the order of their lengths
  int max_len, npages;
  float scale_log2;               // |scale| log2(e)
  float sign;                     // sign of the scale
  const void* q;
  void* out;
  const int32_t *seq_lens, *draft_lens;
  const uint64_t* mask;
  const int32_t *perm, *table;
  int page, max_pages;
  uint32_t page_inv;              // 2^32 / page, rounded down
  float* part;                    // [B Hkv R][nsplit][128] rotated partial results
  float2* ml;                     // [B Hkv R][nsplit] (maximum in log2, sum)
  uint64_t wait;                  // limit of a wait, in SM cycles
  int stall;                      // test hook: the products first wait for a barrier that nothing arrives on
  int* err;
};

// Four consecutive channels 4 lane .. of an output row, or (perm: the kv head's permutation) the
// channels that the row's group coordinates 4 lane .. stand for.
template <typename T>
__device__ __forceinline__ void store_row(T* row, const int32_t* perm, int lane, float4 v) {
  Vec<T, 4> x;
  x.v[0] = from_f<T>(v.x);
  x.v[1] = from_f<T>(v.y);
  x.v[2] = from_f<T>(v.z);
  x.v[3] = from_f<T>(v.w);
  if (!perm) {
    *reinterpret_cast<Vec<T, 4>*>(row + 4 * lane) = x;
    return;
  }
  const int4 to = __ldg(reinterpret_cast<const int4*>(perm) + lane);
  if (to.x >= 0 && to.x < kTD) row[to.x] = x.v[0];
  if (to.y >= 0 && to.y < kTD) row[to.y] = x.v[1];
  if (to.z >= 0 && to.z < kTD) row[to.z] = x.v[2];
  if (to.w >= 0 && to.w < kTD) row[to.w] = x.v[3];
}
// 16 bytes from global to shared memory, asynchronously
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;\n" ::: "memory"); }

__device__ __forceinline__ uint32_t h2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// (a.x s + t, a.y s + t) and pairwise sums, two lanes of 32 bits an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 s, float2 t) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&s)),
        "l"(*reinterpret_cast<const uint64_t*>(&t)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Exponent e in [-110, 110] that brings a row's largest element near 2^9, so that its fp16 operand keeps
// eleven bits of whatever counts in the row (fp16 alone has a fixed step below 6e-5); 2^e as a float.
__device__ __forceinline__ int row_exp(float mx) {
  return mx > 0.f && mx < INFINITY ? max(-110, min(110, 136 - (int)(__float_as_uint(mx) >> 23))) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Tokens of sequence b and the drafted ones among them.
__device__ __forceinline__ void lens_of(const TreeArgs& A, int b, int& len, int& nd) {
  len = max(0, min(A.seq_lens[b], A.max_len));
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

// Every n-th 16-byte piece of a square fp16 matrix of width 64 or 128, into swizzled blocks of 64
// columns with 128-byte rows.  (Rolled: code that runs once a CTA must not push the loops out of the
// instruction cache.  With everything unrolled the kernel had 144 KB of code, and took 748 us where the rolled one took 543.)
template <int W>
__device__ __forceinline__ void copy_matrix(uint8_t* dst, const __half* src, int t, int nt) {
#pragma unroll 1
  for (int e = t; e < W * W / 8; e += nt) {
    const int r = e / (W / 8), c = e % (W / 8);
    copy16(dst + (c >> 3) * W * 128 + swz(r, c & 7), src + (size_t)e * 8);
  }
}

// Bounded wait for an mbarrier phase, compact: it is inlined many times.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, int parity, const volatile int* abort, uint64_t limit) {
  const uint32_t p = (uint32_t)parity & 1u;
  if (mbar_try_wait(bar, p)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try_wait(bar, p))
    if (*abort || (uint64_t)(clock64() - t0) > limit) return false;
  return true;
}

// The code words of one thread's 64 coordinates (two 32-coordinate groups of P words).
// (volatile: the compiler would move a plain load down to its use, behind the waits that it is to overlap)
__device__ __forceinline__ uint4 ld_ahead16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_ahead8(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
// (into a 32-bit register: widening a 16-bit one would wait for the load on the spot)
__device__ __forceinline__ uint32_t ld_ahead2(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u16 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
template <int P>
__device__ __forceinline__ void load_words(uint32_t (&x)[8], const uint8_t* rec) {
  if constexpr (P == 3) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint2 v = ld_ahead8(rec + 8 * i);
      x[2 * i] = v.x;
      x[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const uint4 v = ld_ahead16(rec + 16 * i);
      x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
    }
  }
}
// Byte-permute selectors (low code bits) of slice u of the first group, and its top bits at byte msbs.
template <int P>
__device__ __forceinline__ uint32_t low_sel(const uint32_t (&x)[P], int u) {
  if constexpr (P == 4) return x[u] & 0x77777777u;
  else if constexpr (P == 3) return (x[u & 1] >> (2 * (u >> 1))) & 0x33333333u;
  else return (x[0] >> u) & 0x11111111u;
}
template <int P>
__device__ __forceinline__ uint32_t top_bits(const uint32_t (&x)[P], int u, int h) {
  if constexpr (P == 4) return h ? x[u] << 4 : x[u];
  else return x[P - 1] << (2 * u + h);
}

// 16 bytes to shared memory at address `at` + `off`.
template <int off>
__device__ __forceinline__ void store16(uint32_t at, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0 + %1], {%2, %3, %4, %5};\n" ::"r"(at), "n"(off), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
// Key rows: levels times the norm, and the residual signs times both norms.  `at`: shared address of the
// row's first piece, swizzled (piece c of the row lies at `at` ^ 16 c).  (The loop over the
// two groups is not unrolled: the warps of a CTA run different code, and short loops keep it in
// the instruction cache.)
template <int P>
__device__ __forceinline__ void decode_keys(const uint32_t (&x)[8], const TreeGroup& t, float n, float rn, uint32_t at) {
  const uint32_t nn = h2_bits(n, n);
  // the bytes of +-||k|| ||r||; a set sign bit turns it positive
  const uint32_t rr = h2_bits(n * rn, n * rn);
  const uint32_t rl = prmt(rr, 0u, 0x0000u), rh = prmt(rr, 0u, 0x1111u) | 0x80808080u;
  uint32_t y[P];
#pragma unroll
  for (int i = 0; i < P; ++i) y[i] = x[i];
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t sel = low_sel<P>(y, u);
      uint32_t o[4], s[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sl = h ? sel >> 16 : sel;
        const uint32_t lb = prmt(t.klo[0], t.klo[1], sl), hb = prmt(t.khi[0], t.khi[1], sl);
        o[2 * h] = mul_h2(prmt(lb, hb, 0x5140u), nn);
        o[2 * h + 1] = mul_h2(prmt(lb, hb, 0x7362u), nn);
        const uint32_t sb = (top_bits<P>(y, u, h) & 0x80808080u) ^ rh;
        s[2 * h] = prmt(rl, sb, 0x5140u);
        s[2 * h + 1] = prmt(rl, sb, 0x7362u);
      }
      store16<0>(at ^ (uint32_t)(16 * u), o);
      store16<2 * kTileTok * 128>(at ^ (uint32_t)(16 * u), s);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = x[P + i];
    at ^= 64u;                      // the second group's pieces
  }
}
// Value rows: levels times the norm.
template <int P>
__device__ __forceinline__ void decode_values(const uint32_t (&x)[8], const TreeGroup& t, float n, uint32_t at) {
  const uint32_t nn = h2_bits(n, n);
  uint32_t y[P];
#pragma unroll
  for (int i = 0; i < P; ++i) y[i] = x[i];
#pragma unroll 1
  for (int g = 0; g < 2; ++g) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t sel = low_sel<P>(y, u);
      uint32_t o[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t sl = h ? sel >> 16 : sel;
        const uint32_t lb = prmt(t.vlo[0], t.vlo[1], sl);
        const uint32_t hb = prmt(t.vhi[0], t.vhi[1], sl) ^ (top_bits<P>(y, u, h) & 0x80808080u);
        o[2 * h] = mul_h2(prmt(lb, hb, 0x5140u), nn);
        o[2 * h + 1] = mul_h2(prmt(lb, hb, 0x7362u), nn);
      }
      store16<0>(at ^ (uint32_t)(16 * u), o);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = x[P + i];
    at ^= 64u;                      // the second group's pieces
  }
}

// The same for two barriers, looked at in one go.
__device__ __forceinline__ bool bar_wait2(uint64_t* a, int pa, uint64_t* b, int pb, const volatile int* abort, uint64_t limit) {
  const bool ra = mbar_try_wait(a, (uint32_t)pa & 1u), rb = mbar_try_wait(b, (uint32_t)pb & 1u);
  return __all_sync(0xffffffffu, (ra && rb) || (bar_wait(a, pa, abort, limit) && bar_wait(b, pb, abort, limit))) != 0;
}

struct Bars {
  uint64_t proj, klast, wfull, xfull, ofull, dfull, drain, never;
  // of a stage: K decoded, S formed (so K is free), V decoded, O += P V done (so V and P are free), P formed
  uint64_t kfull[kStages], sfull[kStages], vfull[kStages], vempty[kStages], pfull[kStages];
};

// One decoder thread: token `row` and one half of the head, of tiles set, set + 3, ...  Its code
// words and norms of the next tile come from memory while it decodes this one.
struct Decoder {
  uint32_t kw[8], vw[8];
  uint32_t kn, kr, vn;
  uint32_t slot;                // of the next tile's token; past the end, of any token of the sequence
  bool live;                    // not past the end (else the token's norms count as 0; nothing here depends on a
                                // loaded value before the tile is decoded, which would wait for the load)
  int tok, po, pg;              // the token after that: offset in its page, page
};

template <int PK, int PV, bool TWO>
struct Decode {
  // bytes of a record, and of a half's part of it
  static constexpr int kRec = TWO ? PK * 8 : PK * 16, vRec = TWO ? PV * 8 : PV * 16;
  static constexpr int kPart = TWO ? 0 : PK * 8, vPart = TWO ? 0 : PV * 8;

  __device__ static __forceinline__ void load_k(Decoder& x, const TreeGroup& g, int half) {
    load_words<PK>(x.kw, g.kcodes + (uint64_t)x.slot * kRec + half * kPart);
    x.kn = ld_ahead2(g.knorm + x.slot);
    x.kr = ld_ahead2(g.krnorm + x.slot);
  }
  __device__ static __forceinline__ void load_v(Decoder& x, const TreeGroup& g, int half) {
    load_words<PV>(x.vw, g.vcodes + (uint64_t)x.slot * vRec + half * vPart);
    x.vn = ld_ahead2(g.vnorm + x.slot);
  }
  // Page entry and offset of token x.tok.
  __device__ static __forceinline__ void locate(Decoder& x, const TreeArgs& A, int b) {
    if (!A.table) return;
    int pi = (int)__umulhi((uint32_t)x.tok, A.page_inv);      // x.tok / page, or one less
    x.po = x.tok - pi * A.page;
    if (x.po >= A.page) { x.po -= A.page; ++pi; }
    x.pg = __ldg(A.table + (size_t)b * A.max_pages + pi);
  }
  // Slot of token x.tok, and on to the set's next token; the page entry of a call is loaded by the
  // call before.
  __device__ static __forceinline__ void advance(Decoder& x, const TreeArgs& A, int b, int hk, int t1) {
    x.live = x.tok < t1;
    if (!x.live) return;
    if (A.table) {
      if ((unsigned)x.pg >= (unsigned)A.npages) {
        if (A.err) atomicCAS(A.err, 0, (int)kErrSlotRange);
        x.pg = 0;
      }
      x.slot = (uint32_t)((x.pg * A.Hkv + hk) * A.page + x.po);
    } else {
      x.slot = (uint32_t)((b * A.Hkv + hk) * A.max_len + x.tok);
    }
    x.tok += kSets * kTileTok;
    if (x.tok < t1) locate(x, A, b);
  }
  __device__ static __forceinline__ void start(Decoder& x, const TreeArgs& A, const TreeGroup& g, int half, int tok, int b,
                                               int hk, int t1) {
    x.tok = min(tok, t1 - 1);
    x.po = x.pg = 0;
    locate(x, A, b);
    advance(x, A, b, hk, t1);
    x.live = tok < t1;
    load_k(x, g, half);
    load_v(x, g, half);
  }
  __device__ static __forceinline__ bool loop(Decoder& x, const TreeArgs& A, const TreeGroup& g, uint8_t* smem, Bars* bar,
                                              int half, int set, int row, int b, int hk, int t1, int n,
                                              const volatile int* abort_v, int& code) {
    // the row's first piece of a stage, swizzled
    const uint32_t at0 = (smem_u32(smem) + half * (kTileTok * 128) + row * 128) ^ ((row & 7) << 4);
    const bool lane0 = (threadIdx.x & 31) == 0;
    auto wait = [&](uint64_t* p, int parity) {
      return __all_sync(0xffffffffu, bar_wait(p, parity, abort_v, A.wait)) != 0;
    };
    auto f = [](uint32_t h) { return __half2float(__ushort_as_half((unsigned short)h)); };
#pragma unroll 1
    for (int i = set; i < n; i += kSets) {
      const int st = i % kStages, ph = i / kStages;
      const bool live = x.live;
      // A value norm that is not finite would reach every row through 0 * V, rows that do not attend the
      // token among them: the value counts as 0 and the key as NaN, which only the attending rows see.
      const bool bad = (x.vn & 0x7C00u) == 0x7C00u;
      advance(x, A, b, hk, t1);
      if (!wait(&bar->sfull[st], ph + 1)) { code = 601; return false; }
      decode_keys<PK>(x.kw, g, live ? (bad ? NAN : f(x.kn)) : 0.f, live ? f(x.kr) : 0.f, at0 + st * kKBytes);
      load_k(x, g, half);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane0) mbar_arrive(&bar->kfull[st]);
      if (!wait(&bar->vempty[st], ph + 1)) { code = 602; return false; }
      decode_values<PV>(x.vw, g, live && !bad ? f(x.vn) : 0.f, at0 + kOffV + st * kVBytes);
      load_v(x, g, half);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane0) mbar_arrive(&bar->vfull[st]);
    }
    return true;
  }
};

template <int PK0, int PV0, int PK1, int PV1, bool TWO, typename T>
__global__ void __launch_bounds__(kThreads, 1) tree_attn_kernel(const __grid_constant__ TreeArgs A) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bar = reinterpret_cast<Bars*>(smem + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 512 - 8);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* s_scale = reinterpret_cast<float*>(smem + kOffMisc + 512);      // [128] logit scale of a lane's row; at the end, what undoes its output's
  float2* s_ml = reinterpret_cast<float2*>(smem + kOffMisc + 1024);      // [128] the copies' maxima and sums
  // (a shuffle makes the warp's number, and what the products' addresses come from, known to be uniform: the
  // compiler then keeps the operands of the products in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // Blocks go by split, then sequence, then kv head and row tile: the first splits hold the most tokens.
  // When there are more blocks than SMs, sequences go from the longest to the shortest, so that no long
  // block starts last: thread t finds the rank of sequence t.
  const int rt = blockIdx.x % A.tiles_r, hk = blockIdx.x / A.tiles_r % A.Hkv;
  const int sb = blockIdx.x / (A.tiles_r * A.Hkv), split = sb / A.B;
  int b = sb % A.B;
  if (A.sort) {
    int* s_len = reinterpret_cast<int*>(smem);
    const int mine = threadIdx.x < A.B ? A.seq_lens[threadIdx.x] : INT_MIN;
    s_len[threadIdx.x] = mine;
    __syncthreads();
    if (threadIdx.x < A.B) {
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < A.B; ++j) rank += s_len[j] > mine || (s_len[j] == mine && j < (int)threadIdx.x);
      if (rank == b) s_len[kThreads] = threadIdx.x;
    }
    __syncthreads();
    b = s_len[kThreads];
    __syncthreads();
  }
  const int bh = b * A.Hkv + hk;
  const int r0 = rt * kRows;
  const int nrow = min(kRows, A.R - r0);                 // rows of this tile
  // the matrices and rows of the projection are on their way while the lengths come
  copy_matrix<TWO ? 64 : 128>(smem + kOffPi, A.g[0].pi, threadIdx.x, kThreads);
  copy_matrix<TWO ? 64 : 128>(smem + kOffS, A.g[0].st, threadIdx.x, kThreads);
  if (TWO) {
    copy_matrix<64>(smem + kOffPi + 8192, A.g[1].pi, threadIdx.x, kThreads);
    copy_matrix<64>(smem + kOffS + 8192, A.g[1].st, threadIdx.x, kThreads);
  }
  constexpr int kChunks = kTD * (int)sizeof(T) / 16;
#pragma unroll 1
  for (int e = threadIdx.x; e < nrow * kChunks; e += kThreads) {
    const int r = e / kChunks, c = e % kChunks;
    copy16(smem + kOffV + e * 16, static_cast<const uint8_t*>(A.q) + q_row(A, b, hk, r0 + r) * kTD * sizeof(T) + c * 16);
  }
  int len, nd;
  lens_of(A, b, len, nd);
  const int ctx = len - nd;
  const int live = min(nrow, nd * A.rep - r0);           // those of drafted tokens that exist
  const int t0 = split * A.chunk, t1 = min(len, t0 + A.chunk);
  const int32_t* perm = A.perm ? A.perm + (size_t)hk * kTD : nullptr;
  if (live <= 0 || t0 >= t1) {                           // nothing to attend: zeros (the merge writes its own)
    copy_wait();
    if (A.nsplit == 1)
#pragma unroll 1
      for (int r = warp; r < nrow; r += kThreads / 32)
        store_row<T>(static_cast<T*>(A.out) + q_row(A, b, hk, r0 + r) * kTD, nullptr, lane, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  const int n = __shfl_sync(0xffffffffu, (t1 - t0 + kTileTok - 1) / kTileTok, 0);
  const int fold = A.fold, per = kRows / fold;           // copies of the rows, lanes of a copy
  if (threadIdx.x == 0) {
    mbar_init(&bar->proj, 1);
    mbar_init(&bar->klast, 1);
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar->kfull[i], kDecSet);
      mbar_init(&bar->vfull[i], kDecSet);
      mbar_init(&bar->vempty[i], 1);
      mbar_init(&bar->sfull[i], 1);
      mbar_init(&bar->pfull[i], kSoftWarps);
    }
    mbar_init(&bar->wfull, kDecWarps);
    mbar_init(&bar->xfull, kSoftWarps);
    mbar_init(&bar->ofull, kSoftWarps);
    mbar_init(&bar->dfull, 1);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->never, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  const volatile int* abort_v = abort_flag;
  auto fail = [&](int code) {
    atomicExch(abort_flag, 1);
    if (A.err) atomicCAS(A.err, 0, code);
  };
  // the same answer for the whole warp, which the tensor memory accesses behind it need
  auto wait_all = [&](uint64_t* x, int parity) { return __all_sync(0xffffffffu, bar_wait(x, parity, abort_v, A.wait)) != 0; };
  uint32_t tmem = 0;
  // ------------------------------------------------------------------ projection of the rows
  // A warp a row makes fp16 operands of the rows, scaled by a power of two so that the largest element is near 2^9, every copy of them.
  const int dw = warp - kSoftWarps, half = (dw % kDecSet) >> 1, set = dw / kDecSet, drow = 32 * (dw & 1) + lane;
  Decoder dec;
  if (warp >= kSoftWarps && warp < kMmaWarp) {
    const int tok = t0 + set * kTileTok + drow;
    if (!TWO || half == 0) Decode<PK0, PV0, TWO>::start(dec, A, A.g[0], half, tok, b, hk, t1);
    else Decode<PK1, PV1, TWO>::start(dec, A, A.g[1], 1, tok, b, hk, t1);
  }
  bool ok = true;
  {
    copy_wait();
    __syncthreads();
    int4 ch = make_int4(4 * lane, 4 * lane + 1, 4 * lane + 2, 4 * lane + 3);
    if (perm) ch = __ldg(reinterpret_cast<const int4*>(perm) + lane);
    const bool in = (unsigned)ch.x < kTD && (unsigned)ch.y < kTD && (unsigned)ch.z < kTD && (unsigned)ch.w < kTD;
    if (!in && A.err) atomicCAS(A.err, 0, (int)kErrPermRange);
#pragma unroll 1
    for (int r = warp; r < per; r += kThreads / 32) {
      const T* x = reinterpret_cast<const T*>(smem + kOffV) + r * kTD;
      auto get = [&](int c) { return r < live && (unsigned)c < kTD ? to_f<T>(x[c]) : 0.f; };
      const float4 v = make_float4(get(ch.x), get(ch.y), get(ch.z), get(ch.w));
      float mx = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const int e = row_exp(mx);
      const float up = A.sign * pow2(e);
      const uint2 h = make_uint2(h2_bits(v.x * up, v.y * up), h2_bits(v.z * up, v.w * up));
#pragma unroll 1
      for (int c = r; c < kRows; c += per) {
        *reinterpret_cast<uint2*>(smem + (lane >> 4) * (kRows * 128) + swz(c, (lane >> 1) & 7) + 8 * (lane & 1)) = h;
        // (not 0: a column left out is -inf before the scale)
        if (lane == 0) s_scale[c] = fmaxf(A.scale_log2 * pow2(-e), 1e-30f);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    if (warp == kMmaWarp) {
      // D columns 64 j: coordinates 64 j .. of Pi q, then (from 128 on) of kappa S q
      constexpr uint32_t idesc = idesc_f16(kRows, 64, 0) | kMajorN;
      const uint32_t a0 = smem_u32(smem);
#pragma unroll 1
      for (int pj = 0; pj < 4; ++pj) {
        const int part = pj >> 1, j = pj & 1;
#pragma unroll
        for (int ks = 0; ks < (TWO ? 4 : 8); ++ks) {
          const uint32_t a = TWO ? a0 + j * (kRows * 128) + ks * 32 : a0 + (ks >> 2) * (kRows * 128) + (ks & 3) * 32;
          const uint32_t bb = a0 + (part ? kOffS : kOffPi) + j * (TWO ? 8192 : 16384) + ks * 2048;
          mma_ss_warp(tmem + (uint32_t)(kColS + 64 * pj), desc_sw128(a), desc_mn(bb, 8192), idesc, ks ? 1u : 0u);
        }
      }
      mma_commit_warp(&bar->proj);
    }
    if (!wait_all(&bar->proj, 0)) { fail(603); ok = false; }
    tc_fence_after();
    if (ok && warp < 8) {
      // warps 0-3: Pi q to columns 0 .. 63 of Q, warps 4-7: kappa S q to columns 64 .. 127
      const int part = warp >> 2;
      const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32], o[16];
        tmem_ld32(lane_base + (uint32_t)(kColS + 128 * part + 32 * c), v);
        tmem_ld_wait();
        const float inv = part ? 1.f / 16.f : A.g[TWO && c >= 2 ? 1 : 0].kinv;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = h2_bits(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
        tmem_st16(lane_base + (uint32_t)(kColQ + 64 * part + 16 * c), o);
      }
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    ok = *abort_v == 0;
  }

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------------ softmax, thread = lane = row of a copy
    const int r = threadIdx.x % per;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * warp) << 16);
    const bool warp_live = (32 * warp) % per < live;
    const int j = (r0 + r) / A.rep;
    const bool row_live = r < live;
    const float sc = s_scale[threadIdx.x];
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
    const int copy = (32 * warp) / per, c0 = copy * (64 / fold);      // (a warp's lanes are of one copy)
    // sixteen columns of S to eight of P
    auto weights = [&](const uint32_t* s, float2 sc2, float2 base2, float2& sum, uint32_t (&p)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float2 x = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, base2);
        x.x = ex2(x.x);
        x.y = ex2(x.y);
        sum = add2(sum, x);
        p[e] = h2_bits(x.x, x.y);
      }
    };
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int i = 0; ok && i < n; ++i) {
      const int st = i % kStages, ph = i / kStages;
      if (!wait_all(&bar->sfull[st], ph)) { fail(604); ok = false; break; }
      tc_fence_after();
      if (warp_live) {
        // this copy's columns: from c0 on, 64 / fold of them
        const uint32_t col = lane_base + (uint32_t)(kColS + 64 * st);
        uint32_t s[64];
        if (fold == 1) {
          tmem_ld32(col, reinterpret_cast<uint32_t(&)[32]>(s[0]));
          tmem_ld32(col + 32, reinterpret_cast<uint32_t(&)[32]>(s[32]));
        } else {
          tmem_ld16(col + (uint32_t)c0, reinterpret_cast<uint32_t(&)[16]>(s[0]));
          if (fold == 2) tmem_ld16(col + (uint32_t)c0 + 16, reinterpret_cast<uint32_t(&)[16]>(s[16]));
        }
        tmem_ld_wait();
        const int ts = t0 + i * kTileTok;
        if (ts + kTileTok > min(ctx, t1)) {          // a last tile: columns that the row does not attend become -inf
          const uint64_t keep = kept(ts) >> c0;
          auto cut = [&](uint32_t* x, uint32_t bits) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = (bits >> e) & 1 ? x[e] : 0xFF800000u;
          };
          cut(s, (uint32_t)keep);
          if (fold < 4) cut(s + 16, (uint32_t)(keep >> 16));
          if (fold < 2) {
            cut(s + 32, (uint32_t)(keep >> 32));
            cut(s + 48, (uint32_t)(keep >> 48));
          }
        }
        auto most = [&](const uint32_t* x) {
          float a = -INFINITY, z = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            a = max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            z = max3(z, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
          }
          return fmaxf(a, z);
        };
        float mt = most(s);
        if (fold < 4) mt = fmaxf(mt, most(s + 16));
        if (fold < 2) mt = max3(mt, most(s + 32), most(s + 48));
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
          // O rows times f, once the products of the tile before are in (S of tile i - 1 says that those of
          // tile i - 5 are, so the parity is that of tile i - 1)
          if (!wait_all(&bar->vempty[(i - 1) % kStages], (i - 1) / kStages)) { fail(605); ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(lane_base + kColO + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(lane_base + kColO + 16 * c, o);
          }
        }
        const float base = kPShift - (m == -INFINITY ? 0.f : m);
        const float2 sc2 = make_float2(sc, sc), base2 = make_float2(base, base);
        // P of column t lies in half t & 1 of column t / 2; the other copies' columns get zeros
        float2 sum = make_float2(0.f, 0.f);
        uint32_t p[16];
        if (fold == 4) {
          uint32_t z[8], w8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = 0u;
          weights(s, sc2, base2, sum, w8);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c != copy) tmem_st8(col + 8 * c, z);
          tmem_st8(col + 8 * copy, w8);
        } else {
          weights(s, sc2, base2, sum, reinterpret_cast<uint32_t(&)[8]>(p[0]));
          weights(s + 16, sc2, base2, sum, reinterpret_cast<uint32_t(&)[8]>(p[8]));
          tmem_st16(col + (uint32_t)(c0 / 2), p);
          if (fold == 2) {
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = 0u;
          } else {
            weights(s + 32, sc2, base2, sum, reinterpret_cast<uint32_t(&)[8]>(p[0]));
            weights(s + 48, sc2, base2, sum, reinterpret_cast<uint32_t(&)[8]>(p[8]));
          }
          tmem_st16(col + (uint32_t)(16 - c0 / 2), p);
        }
        l += sum.x + sum.y;
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->pfull[st]);
    }
    // the products of the last tiles (as above, the S of a tile says that those four tiles before it are in)
#pragma unroll 1
    for (int i = max(0, n - kStages); ok && i < n; ++i)
      if (!wait_all(&bar->vempty[i % kStages], i / kStages)) { fail(606); ok = false; }
    // weights of the copies: their common maximum and sum
    if (fold > 1) {
      s_ml[threadIdx.x] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->xfull);
      if (ok && !wait_all(&bar->xfull, 0)) { fail(613); ok = false; }
    }
    float L = l, w = 1.f;
    if (fold > 1) {
      float M = -INFINITY;
#pragma unroll 1
      for (int c = r; c < kRows; c += per) M = fmaxf(M, s_ml[c].x);
      L = 0.f;
#pragma unroll 1
      for (int c = r; c < kRows; c += per) {
        const float2 x = s_ml[c];
        if (x.x != -INFINITY) L += ex2(x.x - M) * x.y;
        else L += x.y;                               // 0, or the NaN of a row without a maximum
      }
      w = m == -INFINITY ? 0.f : ex2(m - M);
      m = M;
    }
    if (ok) {
      tc_fence_after();
      if (warp_live) {
        float inv = L > 0.f || L != L ? w / L : 0.f, mx = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(lane_base + kColO + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, fabsf(__uint_as_float(o[e])));
        }
        const int up = row_exp(mx * inv);
        inv *= pow2(up);
        s_scale[threadIdx.x] = pow2(-up);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32], x[16];
          tmem_ld32(lane_base + kColO + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = h2_bits(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          tmem_st16(lane_base + kColS + 16 * c, x);
        }
        tmem_st_wait();
      }
      tc_fence_before();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->ofull);
    if (ok && !wait_all(&bar->dfull, 0)) { fail(607); ok = false; }
    tc_fence_after();
    // the rotated rows of every copy to shared memory
    float* sums = reinterpret_cast<float*>(smem + kOffSum) + threadIdx.x * kSumLd;
    if (ok && warp_live) {
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[16];
        tmem_ld16(lane_base + kColO + 16 * c, o);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<uint4*>(sums + 16 * c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
    }
    if (A.nsplit > 1 && threadIdx.x < nrow)
      A.ml[((size_t)bh * A.R + r0 + threadIdx.x) * A.nsplit + split] = make_float2(m - kPShift, row_live ? L : 0.f);
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------------ decoders
    int code = 0;
    if (ok) {
      if (!TWO || half == 0)
        ok = Decode<PK0, PV0, TWO>::loop(dec, A, A.g[0], smem, bar, half, set, drow, b, hk, t1, n, abort_v, code);
      else
        ok = Decode<PK1, PV1, TWO>::loop(dec, A, A.g[1], smem, bar, 1, set, drow, b, hk, t1, n, abort_v, code);
      if (!ok) fail(code);
    }
    // the value rotation into the first K stage, once the last logits are formed
    if (ok && !wait_all(&bar->klast, 0)) { fail(608); ok = false; }
    if (ok) {
      const int t = threadIdx.x - 32 * kSoftWarps;
      copy_matrix<TWO ? 64 : 128>(smem, A.g[0].piv, t, 32 * kDecWarps);
      if (TWO) copy_matrix<64>(smem + 8192, A.g[1].piv, t, 32 * kDecWarps);
      copy_wait();
      fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->wfull);
  } else {
    // ------------------------------------------------------------------ products
    const uint32_t k0 = smem_u32(smem), v0 = smem_u32(smem + kOffV);
    if (ok && A.stall && !wait_all(&bar->never, 0)) { fail(615); ok = false; }
    constexpr uint32_t id_s = idesc_f16(kRows, kTileTok, 0), id_o = idesc_f16(kRows, kTD, 0) | kMajorN;
#pragma unroll 1
    for (int i = 0; ok && i < n + kAhead; ++i) {
      if (i < n) {
        // S takes the columns of P of four tiles before: its products are in
        const int st = i % kStages, ph = i / kStages;
        if (!bar_wait2(&bar->kfull[st], ph, &bar->vempty[st], ph + 1, abort_v, A.wait)) { fail(609); ok = false; break; }
        tc_fence_after();
        const uint32_t kb = k0 + st * kKBytes, d = tmem + (uint32_t)(kColS + 64 * st);
#pragma unroll 4
        for (int k = 0; k < 16; ++k)
          mma_ts_warp(d, tmem + (uint32_t)(kColQ + 8 * k), desc_sw128(kb + (k >> 2) * (kTileTok * 128) + (k & 3) * 32), id_s, k ? 1u : 0u);
        mma_commit_warp(&bar->sfull[st]);
        if (i == n - 1) mma_commit_warp(&bar->klast);
      }
      if (i >= kAhead) {
        const int p = i - kAhead, st = p % kStages, ph = p / kStages;
        if (!bar_wait2(&bar->vfull[st], ph, &bar->pfull[st], ph, abort_v, A.wait)) { fail(611); ok = false; break; }
        tc_fence_after();
        const uint32_t vb = v0 + st * kVBytes, a = tmem + (uint32_t)(kColS + 64 * st);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ts_warp(tmem + kColO, a + (uint32_t)(8 * k), desc_mn(vb + k * 2048, kTileTok * 128), id_o, p > 0 || k > 0 ? 1u : 0u);
        mma_commit_warp(&bar->vempty[st]);
      }
    }
    if (ok && (!wait_all(&bar->wfull, 0) || !wait_all(&bar->ofull, 0))) { fail(612); ok = false; }
    if (ok) {
      // out = O / l times Pi of the values
      tc_fence_after();
      const uint32_t a = tmem + kColS;
      if (TWO) {
        constexpr uint32_t id = idesc_f16(kRows, 64, 0);
        for (int g = 0; g < 2; ++g)
          for (int k = 0; k < 4; ++k)
            mma_ts_warp(tmem + kColO + 64 * g, a + (uint32_t)(32 * g + 8 * k), desc_sw128(k0 + g * 8192 + k * 32), id, k ? 1u : 0u);
      } else {
        constexpr uint32_t id = idesc_f16(kRows, kTD, 0);
        for (int k = 0; k < 8; ++k)
          mma_ts_warp(tmem + kColO, a + (uint32_t)(8 * k), desc_sw128(k0 + (k >> 2) * (kTD * 128) + (k & 3) * 32), id, k ? 1u : 0u);
      }
      mma_commit_warp(&bar->dfull);
    }
    mma_commit_warp(&bar->drain);
    mbar_wait(&bar->drain, 0, nullptr, kDrainNs);
    __syncwarp();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (*abort_v) return;
  // ------------------------------------------------------------------ the copies' sum, a warp a row
  const float inv = A.g[TWO && lane >= 16 ? 1 : 0].vinv;
#pragma unroll 1
  for (int r = warp; r < nrow; r += kThreads / 32) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < live) {
#pragma unroll 1
      for (int c = r; c < kRows; c += per) {
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + kOffSum) + c * kSumLd + 4 * lane);
        const float f = s_scale[c];
        v = make_float4(fmaf(f, x.x, v.x), fmaf(f, x.y, v.y), fmaf(f, x.z, v.z), fmaf(f, x.w, v.w));
      }
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
    if (A.nsplit > 1)
      *reinterpret_cast<float4*>(A.part + (((size_t)bh * A.R + r0 + r) * A.nsplit + split) * kTD + 4 * lane) = v;
    else
      store_row<T>(static_cast<T*>(A.out) + q_row(A, b, hk, r0 + r) * kTD, perm, lane, v);
  }
}

// Log-sum-exp merge of the splits, one warp per row, lane = 4 channels.
template <typename T>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs A) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)A.B * A.Hkv * A.R) return;
  const int lane = threadIdx.x & 31;
  const int r = (int)(row % A.R), bh = (int)(row / A.R), b = bh / A.Hkv, hk = bh % A.Hkv;
  int len, nd;
  lens_of(A, b, len, nd);
  const int ns = r / A.rep < nd ? (len + A.chunk - 1) / A.chunk : 0;     // splits that hold tokens
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
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
  store_row<T>(static_cast<T*>(A.out) + q_row(A, b, hk, r) * kTD, A.perm ? A.perm + (size_t)hk * kTD : nullptr, lane, a);
}

struct TreeWs {
  size_t part, ml, total;
  int nsplit, chunk;
  bool waves;                     // more blocks than SMs
};

// Splits of the tokens: as many as give the shortest modelled time, in tiles: a CTA takes its tiles
// and kEdge more for its start and end (20,000 cycles, a tile about 1,400); more CTAs than SMs take
// between their share (lengths differ, and a free SM takes the next CTA) and whole waves; splits
// cost a merge launch.
constexpr int kEdge = 14, kMergeTiles = 4, kMaxSplit = 128;

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
    const int64_t all = std::max<int64_t>(1, ctas) * s;
    const double waves = all <= sms ? 1.0 : 0.5 * ((double)((all + sms - 1) / sms) + (double)all / sms);
    const double t = waves * (double)(per + kEdge) + (s > 1 ? kMergeTiles : 0);
    if (t < best_t - 1e-9) {
      best_t = t;
      best = s;
    }
  }
  const int64_t per = (tiles + best - 1) / best;
  w.chunk = (int)(per * kTileTok);
  w.nsplit = (int)((tiles + per - 1) / per);
  w.waves = ctas * w.nsplit > sms;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  w.ml = w.nsplit > 1 ? up((size_t)rows * w.nsplit * kTD * sizeof(float)) : 0;
  w.total = w.nsplit > 1 ? w.ml + up((size_t)rows * w.nsplit * sizeof(float2)) : 256;
  return w;
}

template <int PK0, int PV0, int PK1, int PV1, bool TWO, typename T>
int launch_main(const TreeArgs& A, unsigned ctas, cudaStream_t st) {
  cudaError_t e = ensure_smem_attrs<tree_attn_kernel<PK0, PV0, PK1, PV1, TWO, T>>(kSmem, true);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tree_attn_kernel)");
  tree_attn_kernel<PK0, PV0, PK1, PV1, TWO, T><<<ctas, kThreads, kSmem, st>>>(A);
  count_launch();
  return check_launch("tree_attn_kernel");
}

template <typename T>
int launch_typed(const TreeArgs& A, int G, int key_bits, cudaStream_t st) {
  const unsigned ctas = (unsigned)((int64_t)A.B * A.Hkv * A.tiles_r * A.nsplit);
  int r;
  if (G == 1 && key_bits == 4) r = launch_main<4, 4, 4, 4, false, T>(A, ctas, st);
  else if (G == 1) r = launch_main<3, 3, 3, 3, false, T>(A, ctas, st);
  else if (key_bits == 4) r = launch_main<4, 4, 3, 3, true, T>(A, ctas, st);
  else r = launch_main<3, 3, 2, 2, true, T>(A, ctas, st);
  if (r != TQ_OK || A.nsplit == 1) return r;
  // (launches early; it waits for the partials)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)A.B * A.Hkv * A.R + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<T>, A);
  count_launch();
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(tree_merge_kernel)");
  return check_launch("tree_merge_kernel");
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
  A.sort = W.waves && B > 1 && B <= kThreads;
  A.fold = A.R <= kRows / 4 ? 4 : A.R <= kRows / 2 ? 2 : 1;
  A.nsplit = W.nsplit; A.chunk = W.chunk;
  A.words = (T + 63) / 64;
  A.max_len = (int)max_len;
  A.scale_log2 = fabsf(scale) * 1.4426950408889634f;
  A.sign = scale < 0.f ? -1.f : 1.f;
  A.q = q; A.out = out;
  A.seq_lens = seq_lens; A.draft_lens = draft_lens; A.mask = mask; A.perm = perm; A.table = table;
  A.part = reinterpret_cast<float*>(ws);
  A.ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + W.ml);
  A.wait = 2 * pipeline_wait_ns();      // (1.965 GHz at most: a limit in ns is never cut short)
  A.stall = debug_stall() ? 1 : 0;
  A.err = kctx[0]->dev_err;
  int64_t pool = INT64_MAX;
  for (int g = 0; g < G; ++g) {
    TreeGroup& t = A.g[g];
    t.kcodes = kc[g].codes; t.knorm = kc[g].norm; t.krnorm = kc[g].rnorm; t.vcodes = vc[g].codes; t.vnorm = vc[g].norm;
    const Codebook &kb = kctx[g]->cb, &vb = vctx[g]->cb;
    for (int i = 0; i < kb.K && i < 8; ++i) {
      const uint32_t h = half_bits(kb.cc[i] * kctx[g]->lev_scale);
      t.klo[i / 4] |= (h & 0xFF) << (8 * (i % 4));
      t.khi[i / 4] |= (h >> 8) << (8 * (i % 4));
    }
    for (int i = 0; i < vb.K / 2 && i < 8; ++i) {
      const uint32_t h = half_bits(vb.c[vb.K / 2 + i] * vctx[g]->lev_scale);
      t.vlo[i / 4] |= (h & 0xFF) << (8 * (i % 4));
      t.vhi[i / 4] |= (h >> 8) << (8 * (i % 4));
    }
    t.kinv = 1.f / (16.f * kctx[g]->lev_scale);
    t.vinv = 1.f / (16.f * vctx[g]->lev_scale);
    t.pi = static_cast<const __half*>(kctx[g]->PiT_f16);
    t.st = static_cast<const __half*>(kctx[g]->ST_f16);
    t.piv = static_cast<const __half*>(vctx[g]->PiT_f16);
    pool = std::min(pool, std::min(kc[g].cap, vc[g].cap));
  }
  if (table) {
    A.page = page;
    A.max_pages = (int)(max_len / page);
    A.page_inv = (uint32_t)((1ull << 32) / (uint64_t)page);
    A.npages = (int)(pool / ((int64_t)Hkv * page));
  }
  const int key_bits = kctx[0]->lay.planes;
  if (q_dtype == TQ_DTYPE_F32) return launch_typed<float>(A, G, key_bits, st);
  if (q_dtype == TQ_DTYPE_BF16) return launch_typed<__nv_bfloat16>(A, G, key_bits, st);
  return launch_typed<__half>(A, G, key_bits, st);
}

}  // namespace tq
