// Page bounds of a paged cache's keys, and the selection of the pages that a sparse decode
// step reads.
//
//   bounds[page][kv head] = (lo, hi): element-wise minimum and maximum of the keys appended
//     to the page (the rows that tq_quantize_kv took, before quantization, in their type:
//     no rounding).
//   score(page) = sum over the kv head's query heads h and channels c of
//     max(q_hc lo_c, q_hc hi_c), an upper bound of the summed inner products with any key of
//     the page.  With lo <= hi this is sum_c (q+_c hi_c + q-_c lo_c), q+ and q- the sums of the
//     heads' positive and negative parts: two products a channel, whatever the head count.  The
//     second form is what is computed, and stands for the empty box as well: a channel in which
//     every key was NaN holds (+inf, -inf), and gives -inf, the bound over no key, where the first
//     form would give +inf.
//     Sums run in 64 bits, so that the choice does not hang on a rounding order.
//   selected = the `select` pages with the highest scores (ties to the lower page), the first
//     and last pages of a sequence in any case, in ascending order.
//
// The chosen pages become a block table per (sequence, kv head): page p of kv head hk holds
// slots (p Hkv + hk) page .., so it is page p Hkv + hk of a cache with one kv head, and the
// decode kernels run on B Hkv sequences of one kv head each.  The decode kernel starts early, so
// it waits for this selection before it reads a length or the table.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.cuh"

namespace tq {
namespace {

// ------------------------------------------------------------------------------ bounds
// CTA = one page of one kv head: thread (row group, vector of V channels) folds every
// `groups`-th row, the groups meet in shared memory.  Bound: HBM, the rows are read once; eight rows
// a thread are in flight, and neighbouring CTAs take the heads of one page, whose rows lie together.
// 131,072 tokens of 8 heads (bf16, 277 MB with the bounds written): 47 us, 5.9 TB/s, 0.90 of a copy's rate;
// one token for each of 64 sequences: 3.9 us.
constexpr int kBoundThreads = 128, kBoundRows = 8, kBoundCtas = 8;   // CTAs an SM

struct BoundArgs {
  const void* k;
  int64_t n;                 // its rows
  int64_t kt, kh;            // strides in elements: token, kv head
  void* bounds;              // [pages][Hkv][2][D]
  const int32_t* cu_new;     // [B + 1] first new row of every sequence
  const int32_t* start;      // [B] tokens of the sequence before the new ones
  const int32_t* table;      // [B][max_pages]
  int Hkv, D, page, max_pages;
  int64_t npages;
};

// a = min or max of a and b, element by element (a NaN gives way); 16-bit types two at a time.
template <bool MAX, typename T, int V>
__device__ __forceinline__ void fold(Vec<T, V>& a, const Vec<T, V>& b) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    T2* x = reinterpret_cast<T2*>(a.v);
    const T2* y = reinterpret_cast<const T2*>(b.v);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) x[j] = MAX ? __hmax2(x[j], y[j]) : __hmin2(x[j], y[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = to_f<T>(a.v[j]), w = to_f<T>(b.v[j]);
      a.v[j] = from_f<T>(MAX ? fmaxf(u, w) : fminf(u, w));
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kBoundThreads, kBoundCtas) page_bounds_kernel(const __grid_constant__ BoundArgs A) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  using VT = Vec<T, V>;
  VT* s_red = reinterpret_cast<VT*>(s_raw);      // [groups][2][lanes]
  const int b = blockIdx.z, hk = blockIdx.x % A.Hkv, first = blockIdx.x / A.Hkv, step = gridDim.x / A.Hkv;
  const int lanes = A.D / V, groups = max(1, kBoundThreads / lanes);
  const int64_t r0 = A.cu_new[b], nnew = (int64_t)A.cu_new[b + 1] - r0;
  if (nnew <= 0 || r0 < 0 || r0 + nnew > A.n) return;
  const int64_t t0 = A.start[b], t1 = t0 + nnew;
  if (t0 < 0) return;
  const int64_t last = min((t1 - 1) / A.page, (int64_t)A.max_pages - 1);
  const int32_t* table = A.table + (size_t)b * A.max_pages;
  int64_t p = t0 / A.page + first;
  int next = p <= last ? table[p] : 0;           // (a page's entry comes while the page before it is folded)
  for (; p <= last; p += step) {
    const int phys = next;
    if (p + step <= last) next = table[p + step];
    if (phys < 0 || phys >= A.npages) continue;   // (the same for the whole CTA)
    const int64_t a = max(t0, p * A.page), e = min(t1, (p + 1) * A.page);
    const int g = threadIdx.x / lanes;
    for (int c = threadIdx.x % lanes; c < lanes && g < groups; c += kBoundThreads) {
      VT lo, hi;
#pragma unroll
      for (int j = 0; j < V; ++j) { lo.v[j] = from_f<T>(INFINITY); hi.v[j] = from_f<T>(-INFINITY); }
      const T* src = static_cast<const T*>(A.k) + (r0 + (a - t0)) * A.kt + hk * A.kh + (int64_t)c * V;
      const int rows = (int)(e - a);
      for (int r = g; r < rows; r += kBoundRows * groups) {
        VT x[kBoundRows];
#pragma unroll
        for (int i = 0; i < kBoundRows; ++i)     // (past the end: the last row again)
          x[i] = *reinterpret_cast<const VT*>(src + (int64_t)min(r + i * groups, rows - 1) * A.kt);
#pragma unroll
        for (int i = 0; i < kBoundRows; ++i) {
          fold<false>(lo, x[i]);
          fold<true>(hi, x[i]);
        }
      }
      s_red[(g * 2) * lanes + c] = lo;
      s_red[(g * 2 + 1) * lanes + c] = hi;
    }
    __syncthreads();
    VT* dst = reinterpret_cast<VT*>(static_cast<T*>(A.bounds) + ((size_t)phys * A.Hkv + hk) * 2 * A.D);
    for (int c = threadIdx.x; c < 2 * lanes; c += kBoundThreads) {
      VT x = s_red[c];
      const bool top = c >= lanes;
      for (int k = 1; k < groups; ++k) {
        if (top) fold<true>(x, s_red[2 * k * lanes + c]);
        else fold<false>(x, s_red[2 * k * lanes + c]);
      }
      if (a > p * A.page) {           // the page held tokens before this call
        if (top) fold<true>(x, dst[c]);
        else fold<false>(x, dst[c]);
      }
      dst[c] = x;
    }
    __syncthreads();
  }
}

template <typename T>
int launch_bounds_t(const BoundArgs& A, int vec, dim3 grid, cudaStream_t st) {
  const int lanes = A.D / vec, groups = std::max(1, kBoundThreads / lanes);
  const size_t sm = (size_t)groups * 2 * A.D * sizeof(T);
  if (vec > 1) page_bounds_kernel<T, 16 / (int)sizeof(T)><<<grid, kBoundThreads, sm, st>>>(A);
  else page_bounds_kernel<T, 1><<<grid, kBoundThreads, sm, st>>>(A);
  count_launch();
  return check_launch("page_bounds_kernel");
}

// ------------------------------------------------------------------------------ scores
// CTA = (sequence, kv head, 16 `batches` pages), 4 warps: q+ and q- of the group are summed once into
// shared memory; a warp takes four pages at a time, whose bounds are all loaded before the first is summed
// (lanes 0-15 the minima, 16-31 the maxima, 8 channels each; twice for 32-bit bounds).  Bound: HBM, 4 D bytes
// a page and head at 16 bits, and before that the latency of the page table and the bounds.
constexpr int kScoreThreads = 128, kScoreCtas = 7, kScoreWarpPages = 4, kScoreBatches = 8;   // (CTAs an SM; batches at most)
constexpr int kSelD = 128;                 // head dimension of the caches that the decode kernels read

struct SelectArgs {
  const void* q;             // [B][Hq][D]
  const void* bounds;        // [pages][Hkv][2][D]
  const int32_t* seq_lens;
  const int32_t* table;      // [B][max_pages]
  int B, Hq, Hkv, D, page, max_pages;
  int64_t max_len, npages, pool;   // pages of the bounds, pages of the caches
  int select, first, last;
  int staged;                // pages whose keys fit into shared memory
  int batches;               // of four pages, for a warp of the scores
  uint64_t* key;             // [B Hkv][max_pages] order-preserving scores
  int32_t* selected;         // [B][Hkv][select] or NULL
  int32_t* vtable;           // [B Hkv][select] pages of the one-head view
  int32_t* vlen;             // [B Hkv] tokens of the selected pages
};

__device__ __forceinline__ int live_tokens(const SelectArgs& A, int b) {
  return max(0, (int)min((int64_t)A.seq_lens[b], A.max_len));
}

// Unsigned integers in the order of the scores; a NaN comes last.
__device__ __forceinline__ uint64_t order_key(double s) {
  if (s != s) return 0;
  const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);   // (-0 becomes +0)
  return (u >> 63) ? ~u : u | (1ull << 63);
}

__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <typename TQ, typename TB>
__global__ void __launch_bounds__(kScoreThreads, sizeof(TB) == 4 ? 5 : kScoreCtas) page_score_kernel(const __grid_constant__ SelectArgs A) {
  __shared__ double s_q[2 * kSelD];   // sums of the heads' negative parts (for the minima), then of the positive ones
  const int hk = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dep_launch();
  const int mine = kScoreWarpPages * A.batches;                // pages of a warp (32 at most)
  const int p0 = (blockIdx.x * (kScoreThreads / 32) + warp) * mine;
  const int rep = A.Hq / A.Hkv;
  constexpr int kV = 16 / (int)sizeof(TB), kL = 8 / kV;       // channels a load, loads a lane
  using VT = Vec<TB, kV>;
  int phys = -1;                                              // of page p0 + lane
  if (lane < mine && p0 + lane < A.max_pages) phys = A.table[(size_t)b * A.max_pages + p0 + lane];
  const int n = (live_tokens(A, b) + A.page - 1) / A.page;
  if (p0 + lane >= n) phys = -1;
  VT box[kScoreWarpPages][kL];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kScoreWarpPages; ++i) {
      const int pg = __shfl_sync(0xffffffffu, phys, i0 + i);
      const bool in = pg >= 0 && pg < A.npages;
      const TB* src = static_cast<const TB*>(A.bounds) + ((size_t)(in ? pg : 0) * A.Hkv + hk) * 2 * kSelD + 8 * lane;
#pragma unroll
      for (int j = 0; j < kL; ++j)
        if (in) box[i][j] = *reinterpret_cast<const VT*>(src + j * kV);
    }
  };
  fetch(0);
  {
    static_assert(kScoreThreads == kSelD, "a thread a channel");
    double pos = 0.0, neg = 0.0;
    const TQ* q = static_cast<const TQ*>(A.q) + ((size_t)b * A.Hq + (size_t)hk * rep) * kSelD + threadIdx.x;
#pragma unroll 4
    for (int h = 0; h < rep; ++h) {
      const float v = to_f<TQ>(q[(size_t)h * kSelD]);
      if (v > 0.f) pos += v;
      else neg += v;                 // (a NaN makes the score NaN)
    }
    s_q[threadIdx.x] = neg;
    s_q[kSelD + threadIdx.x] = pos;
  }
  __syncthreads();
  double q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = s_q[8 * lane + j];
  uint32_t keep[kL * 4];              // bits of the channels whose q is not 0: 0 * infinity is no bound
#pragma unroll
  for (int w = 0; w < kL * 4; ++w)
    keep[w] = kL == 2 ? (q[w] != 0.0 ? ~0u : 0u)
                      : (q[2 * w % 8] != 0.0 ? 0xFFFFu : 0u) | (q[(2 * w + 1) % 8] != 0.0 ? 0xFFFF0000u : 0u);
#pragma unroll 1
  for (int i0 = 0; i0 < mine && p0 + i0 < n; i0 += kScoreWarpPages) {
    if (i0 > 0) fetch(i0);
    double s[kScoreWarpPages];
#pragma unroll
    for (int i = 0; i < kScoreWarpPages; ++i) {
      const int pg = __shfl_sync(0xffffffffu, phys, i0 + i);
      s[i] = 0.0;
      if (pg >= 0 && pg < A.npages) {
        uint32_t* w = reinterpret_cast<uint32_t*>(box[i]);
#pragma unroll
        for (int j = 0; j < kL * 4; ++j) w[j] &= keep[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i] = fma(q[j], (double)to_f<TB>(box[i][j / kV].v[j % kV]), s[i]);
      } else {
        s[i] = -INFINITY;
      }
    }
    // sums over the lanes: halves of the warp take two pages each, then quarters one
    const bool up = lane & 16, up2 = lane & 8;
    double x0 = up ? s[2] : s[0], x1 = up ? s[3] : s[1];
    x0 += __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
    x1 += __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 16);
    double x = up2 ? x1 : x0;
    x += __shfl_xor_sync(0xffffffffu, up2 ? x0 : x1, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const int p = p0 + i0 + (lane >> 3);
    if ((lane & 7) == 0 && p < n) {
      uint64_t key = order_key(x);
      if (key == ~0ull) --key;
      if (p < A.first || p >= n - A.last) key = ~0ull;
      A.key[((size_t)b * A.Hkv + hk) * A.max_pages + p] = key;
    }
  }
  dep_wait();     // (the projection of the queries in front of this kernel is done when this one is)
}

// ------------------------------------------------------------------------------ selection
// CTA per (sequence, kv head); keys sit in shared memory when they fit.  Two ways:
//   few pages: every page counts the keys in front of it;
//   many: the select-th largest key by 8-bit digits (a histogram of the keys that share the prefix found so
//     far, from the highest bit in which any two keys differ on), then one ordered pass that keeps the larger
//     keys and the first of the equal ones.
// Bound: latency (the keys are a few KB).  The whole sparse step of 4 sequences x 8 kv heads took, in us,
//   pages      64    128    192    256    512
//   counted  27.7   28.7   30.3   31.3   40.9     (n^2 comparisons of 64 bits: several lanes a page change nothing)
//   digits   29.5   29.8   29.8   29.9   30.3
constexpr int kSelThreads = 512, kSelStaged = 4096, kSelRank = 160;

__global__ void __launch_bounds__(kSelThreads) page_pick_kernel(const __grid_constant__ SelectArgs A) {
  extern __shared__ __align__(16) uint64_t s_key[];
  __shared__ int hist[256];
  __shared__ int s_warp[kSelThreads / 32][2];
  __shared__ uint64_t s_and[kSelThreads / 32], s_or[kSelThreads / 32];
  __shared__ uint64_t s_prefix;
  __shared__ int s_need, s_done;
  const int vh = blockIdx.x, b = vh / A.Hkv, hk = vh % A.Hkv;
  const int len = live_tokens(A, b), n = (len + A.page - 1) / A.page;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t* table = A.table + (size_t)b * A.max_pages;
  auto view = [&](int i) {           // page i as a page of the one-head view
    const int phys = table[i];
    return phys >= 0 && phys < A.pool ? phys * A.Hkv + hk : -1;
  };
  int ahead = n > A.select && tid < n ? view(tid) : -1;     // (on its way while the scores are formed)
  dep_wait();                        // the scores
  if (n <= A.select) {               // every page
    for (int i = tid; i < A.select; i += kSelThreads) {
      if (A.selected) A.selected[(size_t)vh * A.select + i] = i < n ? i : -1;
      A.vtable[(size_t)vh * A.select + i] = i < n ? view(i) : -1;
    }
    if (tid == 0) A.vlen[vh] = len;
    return;
  }
  const uint64_t* gkey = A.key + (size_t)vh * A.max_pages;
  if (n <= kSelRank) {
    // few pages: every page counts the pages in front of it
    const int all = (n + 1) & ~1;
    for (int i = tid; i < all; i += kSelThreads) s_key[i] = i < n ? gkey[i] : 0;
    __syncthreads();
    bool take = false;
    if (tid < n) {
      const uint64_t k = s_key[tid];
      int front = 0;
#pragma unroll 4
      for (int j = 0; j < all; j += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s_key + j);
        front += o.x > k || (o.x == k && j < tid);
        front += o.y > k || (o.y == k && j + 1 < tid);
      }
      take = front < A.select;
    }
    const unsigned tm = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[warp][0] = __popc(tm);
    __syncthreads();
    int rank = __popc(tm & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) rank += s_warp[w][0];
    if (take) {
      if (A.selected) A.selected[(size_t)vh * A.select + rank] = tid;
      A.vtable[(size_t)vh * A.select + rank] = ahead;
      if (rank == A.select - 1) A.vlen[vh] = tid == n - 1 ? (A.select - 1) * A.page + (len - tid * A.page) : A.select * A.page;
    }
    return;
  }
  const bool staged = n <= A.staged;
  uint64_t all_and = ~0ull, all_or = 0;
  for (int i0 = tid; i0 < n; i0 += 4 * kSelThreads) {
    uint64_t k[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = i0 + j * kSelThreads < n ? gkey[i0 + j * kSelThreads] : ~0ull;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (staged && i0 + j * kSelThreads < n) s_key[i0 + j * kSelThreads] = k[j];
      if (k[j] != ~0ull) { all_and &= k[j]; all_or |= k[j]; }     // (the pages taken in any case have no score)
    }
  }
  const uint64_t* key = staged ? s_key : gkey;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all_and &= __shfl_xor_sync(0xffffffffu, all_and, o);
    all_or |= __shfl_xor_sync(0xffffffffu, all_or, o);
  }
  if (lane == 0) { s_and[warp] = all_and; s_or[warp] = all_or; }
  __syncthreads();
  for (int w = 0; w < kSelThreads / 32; ++w) { all_and &= s_and[w]; all_or |= s_or[w]; }
  // keys above `bar` are taken, and the first `need` keys equal to it; forced pages (all ones) first
  int forced = 0;
  {
    const int last = max(0, n - A.last);
    forced = min(n, A.first) + n - max(last, min(n, A.first));
  }
  const int want = A.select;
  uint64_t bar = ~0ull, mask = ~0ull;
  int need = want;                   // (more pages forced than wanted: the first of them)
  if (forced < want) {
    const uint64_t diff = all_and ^ all_or;
    const int high = diff ? 63 - __clzll((long long)diff) : 0;
    int shift = max(0, high - 7);    // the first digit
    if (tid == 0) { s_prefix = high + 1 < 64 ? all_and & (~0ull << (high + 1)) : 0; s_need = want - forced; s_done = 0; }
    int width = high + 1 - shift;    // bits of the digit
    for (;;) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint64_t prefix = s_prefix;
      const uint64_t above = shift + width < 64 ? ~0ull << (shift + width) : 0;
      const uint32_t digits = (1u << width) - 1;
      for (int i = tid; i < n; i += kSelThreads) {
        const uint64_t k = key[i];
        if (k != ~0ull && (k & above) == prefix) atomicAdd(&hist[(uint32_t)(k >> shift) & digits], 1);
      }
      __syncthreads();
      if (warp == 0) {                // digit of the need-th largest key with this prefix
        const int left = s_need;
        int sum = 0, mine[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) { mine[j] = hist[255 - (lane * 8 + j)]; sum += mine[j]; }
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        before -= sum;                // keys in larger digits
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (before < left && before + mine[j] >= left) {
            s_prefix = prefix | ((uint64_t)(255 - (lane * 8 + j)) << shift);
            s_need = left - before;
            s_done = mine[j] == left - before;   // the whole digit is taken: no further digit decides
          }
          before += mine[j];
        }
      }
      __syncthreads();
      if (s_done || shift == 0) break;
      width = min(8, shift);
      shift -= width;
    }
    bar = s_prefix;
    need = s_need;
    mask = ~0ull << shift;            // (keys are compared by their digits from `shift` on)
  }
  int base = 0, eq_base = 0;
  for (int i0 = 0; i0 < n && base < want; i0 += kSelThreads) {
    const int i = i0 + tid, here = ahead;
    if (i + kSelThreads < n) ahead = view(i + kSelThreads);
    const uint64_t k = i < n ? key[i] : 0;
    const bool must = forced < want && k == ~0ull;
    const bool gt = must || (i < n && (k & mask) > bar), eq = !gt && i < n && (k & mask) == bar;
    const unsigned eqm = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[warp][0] = __popc(eqm);
    __syncthreads();
    int eq_rank = eq_base + __popc(eqm & ((1u << lane) - 1)), eq_all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) eq_rank += s_warp[w][0];
      eq_all += s_warp[w][0];
    }
    const bool take = gt || (eq && eq_rank < need);
    const unsigned tm = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[warp][1] = __popc(tm);
    __syncthreads();
    int rank = base + __popc(tm & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) rank += s_warp[w][1];
      all += s_warp[w][1];
    }
    if (take) {
      if (A.selected) A.selected[(size_t)vh * A.select + rank] = i;
      A.vtable[(size_t)vh * A.select + rank] = here;
      if (rank == want - 1) A.vlen[vh] = i == n - 1 ? (want - 1) * A.page + (len - i * A.page) : want * A.page;
    }
    base += all;
    eq_base += eq_all;
    __syncthreads();
  }
}

// Launch that may start while the kernel in front of it still runs (it waits for what it needs).
template <typename K>
int launch_early(K kern, dim3 grid, int threads, size_t smem, const SelectArgs& A, cudaStream_t st, const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, A);
  count_launch();
  if (e != cudaSuccess) return cuda_fail(e, what);
  return check_launch(what);
}

template <typename TQ>
int launch_score_q(const SelectArgs& A, int bounds_dtype, dim3 grid, cudaStream_t st) {
  if (bounds_dtype == TQ_DTYPE_F32) return launch_early(page_score_kernel<TQ, float>, grid, kScoreThreads, 0, A, st, "page_score_kernel");
  if (bounds_dtype == TQ_DTYPE_BF16)
    return launch_early(page_score_kernel<TQ, __nv_bfloat16>, grid, kScoreThreads, 0, A, st, "page_score_kernel");
  return launch_early(page_score_kernel<TQ, __half>, grid, kScoreThreads, 0, A, st, "page_score_kernel");
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int launch_page_bounds(const void* k, int64_t n, int dtype, int64_t k_token, int64_t k_head, const int32_t* cu_new,
                       const int32_t* start, int B, int Hkv, int D, int64_t max_new, const int32_t* table,
                       int page, int max_pages, void* bounds, int64_t npages, cudaStream_t st) {
  const int es = dtype == TQ_DTYPE_F32 ? 4 : 2;
  BoundArgs A{};
  A.k = k; A.n = n; A.kt = k_token; A.kh = k_head; A.bounds = bounds; A.cu_new = cu_new; A.start = start; A.table = table;
  A.Hkv = Hkv; A.D = D; A.page = page; A.max_pages = max_pages; A.npages = npages;
  const int vec = 16 / es;
  const bool wide = D % vec == 0 && reinterpret_cast<uintptr_t>(k) % 16 == 0 && reinterpret_cast<uintptr_t>(bounds) % 16 == 0 && k_token % vec == 0 && k_head % vec == 0;
  const int64_t touched = std::min<int64_t>(max_pages, (max_new + page - 2) / page + 1);
  // one wave of CTAs: each has pages enough that its first loads (lengths, table) do not count, and none
  // is left for a second, almost empty wave (12 CTAs an SM, of which 9 fit: 77 us for the 128K prompt)
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t ctas = std::max<int64_t>(1, (int64_t)kBoundCtas * sms / ((int64_t)Hkv * B));
  const dim3 grid((unsigned)(std::min<int64_t>(touched, ctas) * Hkv), 1, (unsigned)B);
  const int v = wide ? vec : 1;
  if (dtype == TQ_DTYPE_F32) return launch_bounds_t<float>(A, v, grid, st);
  if (dtype == TQ_DTYPE_BF16) return launch_bounds_t<__nv_bfloat16>(A, v, grid, st);
  return launch_bounds_t<__half>(A, v, grid, st);
}

SparseWs sparse_ws(int B, int Hq, int Hkv, int D, int G, int page, int max_pages, int select) {
  SparseWs w{};
  const size_t vh = (size_t)B * Hkv;
  w.key = 0;
  w.vtable = up256(vh * max_pages * sizeof(uint64_t));
  w.vlen = w.vtable + up256(vh * select * sizeof(int32_t));
  w.decode = w.vlen + up256(vh * sizeof(int32_t));
  w.total = w.decode + decode_ws(B * Hkv, Hq / Hkv, 1, D, G, (int64_t)select * page).total;
  return w;
}

int launch_page_select(const void* q, int q_dtype, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                       int64_t max_len, int64_t pool, const tq_sparse_opts* o, void* ws, const SparseWs& W,
                       cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  SelectArgs A{};
  A.q = q; A.bounds = o->bounds; A.seq_lens = seq_lens; A.table = o->block_table;
  A.B = B; A.Hq = Hq; A.Hkv = Hkv; A.D = D; A.page = o->page_tokens; A.max_pages = (int)(max_len / o->page_tokens);
  A.max_len = max_len; A.npages = o->bounds_pages; A.pool = pool;
  A.select = o->select; A.first = o->first; A.last = o->last; A.selected = o->selected;
  A.key = reinterpret_cast<uint64_t*>(base + W.key);
  A.vtable = reinterpret_cast<int32_t*>(base + W.vtable);
  A.vlen = reinterpret_cast<int32_t*>(base + W.vlen);
  int r = TQ_OK;
  if (A.max_pages > A.select) {        // (otherwise every page is read and none is scored)
    // one wave of CTAs, each with as few pages as that allows (32 pages a CTA and several waves: 17.4 us for
    // 64 sequences of 8 heads and 128 pages; so: 12.8 us)
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int step = kScoreWarpPages * (kScoreThreads / 32);
    A.batches = 1;
    while (A.batches < kScoreBatches && (int64_t)div_up(A.max_pages, step * A.batches) * Hkv * B > (int64_t)kScoreCtas * sms) ++A.batches;
    const dim3 grid((unsigned)div_up(A.max_pages, step * A.batches), (unsigned)Hkv, (unsigned)B);
    if (q_dtype == TQ_DTYPE_F32) r = launch_score_q<float>(A, o->bounds_dtype, grid, st);
    else if (q_dtype == TQ_DTYPE_BF16) r = launch_score_q<__nv_bfloat16>(A, o->bounds_dtype, grid, st);
    else r = launch_score_q<__half>(A, o->bounds_dtype, grid, st);
    if (r != TQ_OK) return r;
  }
  A.staged = kSelStaged;
  const size_t sm = A.max_pages > A.select ? (size_t)std::min(A.max_pages + 1, kSelStaged) * sizeof(uint64_t) : 0;
  return launch_early(page_pick_kernel, dim3((unsigned)(B * Hkv)), kSelThreads, sm, A, st, "page_pick_kernel");
}

}  // namespace tq
