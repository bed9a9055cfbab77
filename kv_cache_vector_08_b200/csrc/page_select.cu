// Page bounds of a paged cache's keys, and the selection of the pages that a sparse decode
// step reads.
//
//   bounds[page][kv head] = (lo, hi): element-wise minimum and maximum of the keys appended
//     to the page (the rows that tq_quantize_kv took, before quantization, in their type:
//     no rounding).
//   score(page) = sum over the kv head's query heads h and channels c of
//     max(q_hc lo_c, q_hc hi_c), an upper bound of the summed inner products with any key of
//     the page.  With lo <= hi this is sum_c (q+_c hi_c + q-_c lo_c), q+ and q- the sums of the
//     heads' positive and negative parts: two products a channel, whatever the head count.
//     Sums run in 64 bits, so that the choice does not hang on a rounding order.
//   selected = the `select` pages with the highest scores (ties to the lower page), the first
//     and last pages of a sequence in any case, in ascending order.
//
// The chosen pages become a block table per (sequence, kv head): page p of kv head hk holds
// slots (p Hkv + hk) page .., so it is page p Hkv + hk of a cache with one kv head, and the
// decode kernels run on B Hkv sequences of one kv head each, unchanged.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.cuh"

namespace tq {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// ------------------------------------------------------------------------------ bounds
// CTA = one page of one kv head: thread (row group, vector of V channels) folds every
// `groups`-th row, the groups meet in shared memory.  Bound: HBM, the rows are read once;
// four rows a thread are in flight.
constexpr int kBoundThreads = 128;

struct BoundArgs {
  const void* k;
  int64_t kt, kh;            // strides in elements: token, kv head
  void* bounds;              // [pages][Hkv][2][D]
  const int32_t* cu_new;     // [B + 1] first new row of every sequence
  const int32_t* start;      // [B] tokens of the sequence before the new ones
  const int32_t* table;      // [B][max_pages]
  int Hkv, D, page, max_pages;
  int64_t npages;
};

template <typename T, int V>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const BoundArgs A) {
  extern __shared__ float s_red[];   // [groups][2][D]
  const int b = blockIdx.z, hk = blockIdx.y;
  const int lanes = A.D / V, groups = max(1, kBoundThreads / lanes);
  const int64_t r0 = A.cu_new[b], nnew = (int64_t)A.cu_new[b + 1] - r0;
  if (nnew <= 0) return;
  const int64_t t0 = A.start[b], t1 = t0 + nnew;
  if (t0 < 0) return;
  const int64_t last = min((t1 - 1) / A.page, (int64_t)A.max_pages - 1);
  for (int64_t p = t0 / A.page + blockIdx.x; p <= last; p += gridDim.x) {
    const int phys = A.table[(size_t)b * A.max_pages + p];
    const bool live = phys >= 0 && phys < A.npages;   // (the same for the whole CTA)
    const int64_t a = max(t0, p * A.page), e = min(t1, (p + 1) * A.page);
    T* dst = static_cast<T*>(A.bounds) + ((size_t)(live ? phys : 0) * A.Hkv + hk) * 2 * A.D;
    if (live) {
      const int g = threadIdx.x / lanes;
      for (int c = threadIdx.x % lanes; c < lanes && g < groups; c += kBoundThreads) {
        float lo[V], hi[V];
#pragma unroll
        for (int j = 0; j < V; ++j) { lo[j] = INFINITY; hi[j] = -INFINITY; }
        const T* src = static_cast<const T*>(A.k) + (r0 + (a - t0)) * A.kt + hk * A.kh + (int64_t)c * V;
#pragma unroll 4
        for (int64_t r = g; r < e - a; r += groups) {
          const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(src + r * A.kt);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float f = to_f<T>(x.v[j]);
            lo[j] = fminf(lo[j], f);
            hi[j] = fmaxf(hi[j], f);
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          s_red[(g * 2) * A.D + c * V + j] = lo[j];
          s_red[(g * 2 + 1) * A.D + c * V + j] = hi[j];
        }
      }
    }
    __syncthreads();
    if (live)
      for (int c = threadIdx.x; c < A.D; c += kBoundThreads) {
        float lo = INFINITY, hi = -INFINITY;
        for (int g = 0; g < groups; ++g) {
          lo = fminf(lo, s_red[(g * 2) * A.D + c]);
          hi = fmaxf(hi, s_red[(g * 2 + 1) * A.D + c]);
        }
        if (a > p * A.page) {       // the page held tokens before this call
          lo = fminf(lo, to_f<T>(dst[c]));
          hi = fmaxf(hi, to_f<T>(dst[A.D + c]));
        }
        dst[c] = from_f<T>(lo);
        dst[A.D + c] = from_f<T>(hi);
      }
    __syncthreads();
  }
}

template <typename T>
int launch_bounds_t(const BoundArgs& A, int vec, dim3 grid, cudaStream_t st) {
  const int lanes = A.D / vec, groups = std::max(1, kBoundThreads / lanes);
  const size_t sm = (size_t)groups * 2 * A.D * sizeof(float);
  if (vec > 1) page_bounds_kernel<T, 16 / (int)sizeof(T)><<<grid, kBoundThreads, sm, st>>>(A);
  else page_bounds_kernel<T, 1><<<grid, kBoundThreads, sm, st>>>(A);
  count_launch();
  return check_launch("page_bounds_kernel");
}

// ------------------------------------------------------------------------------ scores
// CTA = (sequence, kv head, kScorePages pages), 8 warps: q+ and q- of the group are summed
// once into shared memory, then a warp takes a page at a time: lane l holds channels
// l, l + 32, ... of both bounds.  Bound: HBM, 4 D bytes a page and head at 16 bits.
constexpr int kScoreThreads = 256, kScorePages = 64;

struct SelectArgs {
  const void* q;             // [B][Hq][D]
  const void* bounds;        // [pages][Hkv][2][D]
  const int32_t* seq_lens;
  const int32_t* table;      // [B][max_pages]
  int B, Hq, Hkv, D, page, max_pages;
  int64_t max_len, npages, pool;   // pages of the bounds, pages of the caches
  int select, first, last;
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

template <typename TQ, typename TB>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectArgs A) {
  extern __shared__ double s_q[];   // [2][D]: sums of the heads' positive and negative parts
  const int hk = blockIdx.y, b = blockIdx.z;
  const int n = (live_tokens(A, b) + A.page - 1) / A.page;
  const int p0 = blockIdx.x * kScorePages, p1 = min(n, p0 + kScorePages);
  if (p0 >= p1) return;
  const int rep = A.Hq / A.Hkv;
  for (int c = threadIdx.x; c < A.D; c += kScoreThreads) {
    double pos = 0.0, neg = 0.0;
    const TQ* q = static_cast<const TQ*>(A.q) + ((size_t)b * A.Hq + (size_t)hk * rep) * A.D + c;
    for (int h = 0; h < rep; ++h) {
      const float v = to_f<TQ>(q[(size_t)h * A.D]);
      if (v > 0.f) pos += v;
      else neg += v;                 // (a NaN makes the score NaN)
    }
    s_q[c] = pos;
    s_q[A.D + c] = neg;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int p = p0 + warp; p < p1; p += kScoreThreads / 32) {
    uint64_t key = ~0ull;
    if (p >= A.first && p < n - A.last) {
      const int phys = A.table[(size_t)b * A.max_pages + p];
      double s = 0.0;
      if (phys >= 0 && phys < A.npages) {
        const TB* box = static_cast<const TB*>(A.bounds) + ((size_t)phys * A.Hkv + hk) * 2 * A.D;
        for (int c = lane; c < A.D; c += 32) {
          const double qp = s_q[c], qn = s_q[A.D + c];
          // a zero part leaves its bound out (0 * infinity is no bound)
          if (qp != 0.0) s += qp * (double)to_f<TB>(box[A.D + c]);
          if (qn != 0.0) s += qn * (double)to_f<TB>(box[c]);
        }
      } else {
        s = -INFINITY;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      key = order_key(s);
      if (key == ~0ull) --key;
    }
    if (lane == 0) A.key[((size_t)b * A.Hkv + hk) * A.max_pages + p] = key;
  }
}

// ------------------------------------------------------------------------------ selection
// CTA per (sequence, kv head): the select-th largest key by 8-bit digits (a histogram of the
// keys that share the prefix found so far, most significant digit first), then one ordered
// pass that keeps the larger keys and the first of the equal ones.
constexpr int kSelThreads = 256;

__global__ void __launch_bounds__(kSelThreads) page_pick_kernel(const SelectArgs A) {
  __shared__ int hist[256];
  __shared__ int s_warp[kSelThreads / 32][2];
  __shared__ uint64_t s_prefix;
  __shared__ int s_need, s_done;
  const int vh = blockIdx.x, b = vh / A.Hkv, hk = vh % A.Hkv;
  const int len = live_tokens(A, b), n = (len + A.page - 1) / A.page;
  const uint64_t* key = A.key + (size_t)vh * A.max_pages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int want = min(A.select, n);
  // keys above `bar` are taken, and the first `need` keys equal to it
  uint64_t bar = 0;
  int need = 0;
  if (n <= A.select) {
    need = n;                         // every page: each key is >= 0, taken by `all` below
  } else {
    if (tid == 0) { s_prefix = 0; s_need = want; s_done = 0; }
    __syncthreads();
    int shift = 56;
    for (; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint64_t prefix = s_prefix;
      const uint64_t above = shift == 56 ? 0 : ~0ull << (shift + 8);
      for (int i = tid; i < n; i += kSelThreads) {
        const uint64_t k = key[i];
        if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
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
      if (s_done) break;
    }
    // every key whose digits from `shift` on are above or equal to the prefix is taken, down
    // to the lowest page; with no digits left, only the first s_need of the equal keys
    bar = s_prefix;
    need = s_need;
    if (shift < 0) shift = 0;
    const uint64_t mask = ~0ull << shift;
    // (below, keys are compared by their digits from `shift` on)
    int base = 0, eq_base = 0;
    for (int i0 = 0; i0 < n; i0 += kSelThreads) {
      const int i = i0 + tid;
      const uint64_t k = i < n ? key[i] & mask : 0;
      const bool gt = i < n && k > bar, eq = i < n && k == bar;
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
        const int phys = A.table[(size_t)b * A.max_pages + i];
        if (A.selected) A.selected[(size_t)vh * A.select + rank] = i;
        A.vtable[(size_t)vh * A.select + rank] = phys >= 0 && phys < A.pool ? phys * A.Hkv + hk : -1;
        if (rank == want - 1) A.vlen[vh] = i == n - 1 ? (want - 1) * A.page + (len - i * A.page) : want * A.page;
      }
      base += all;
      eq_base += eq_all;
      __syncthreads();
    }
    return;
  }
  for (int i = tid; i < A.select; i += kSelThreads) {
    int v = -1;
    if (i < n) {
      const int phys = A.table[(size_t)b * A.max_pages + i];
      if (phys >= 0 && phys < A.pool) v = phys * A.Hkv + hk;
    }
    if (A.selected) A.selected[(size_t)vh * A.select + i] = i < n ? i : -1;
    A.vtable[(size_t)vh * A.select + i] = v;
  }
  if (tid == 0) A.vlen[vh] = len;
}

template <typename TQ>
int launch_score_q(const SelectArgs& A, int bounds_dtype, dim3 grid, cudaStream_t st) {
  const size_t sm = (size_t)2 * A.D * sizeof(double);
  if (bounds_dtype == TQ_DTYPE_F32) page_score_kernel<TQ, float><<<grid, kScoreThreads, sm, st>>>(A);
  else if (bounds_dtype == TQ_DTYPE_BF16) page_score_kernel<TQ, __nv_bfloat16><<<grid, kScoreThreads, sm, st>>>(A);
  else page_score_kernel<TQ, __half><<<grid, kScoreThreads, sm, st>>>(A);
  count_launch();
  return check_launch("page_score_kernel");
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int launch_page_bounds(const void* k, int dtype, int64_t k_token, int64_t k_head, const int32_t* cu_new,
                       const int32_t* start, int B, int Hkv, int D, int64_t max_new, const int32_t* table,
                       int page, int max_pages, void* bounds, int64_t npages, cudaStream_t st) {
  const int es = dtype == TQ_DTYPE_F32 ? 4 : 2;
  BoundArgs A{};
  A.k = k; A.kt = k_token; A.kh = k_head; A.bounds = bounds; A.cu_new = cu_new; A.start = start; A.table = table;
  A.Hkv = Hkv; A.D = D; A.page = page; A.max_pages = max_pages; A.npages = npages;
  const int vec = 16 / es;
  const bool wide = D % vec == 0 && reinterpret_cast<uintptr_t>(k) % 16 == 0 && k_token % vec == 0 && k_head % vec == 0;
  const int64_t touched = std::min<int64_t>(max_pages, (max_new + page - 2) / page + 1);
  const dim3 grid((unsigned)std::min<int64_t>(touched, 65535), (unsigned)Hkv, (unsigned)B);
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
    const dim3 grid((unsigned)div_up(A.max_pages, kScorePages), (unsigned)Hkv, (unsigned)B);
    if (q_dtype == TQ_DTYPE_F32) r = launch_score_q<float>(A, o->bounds_dtype, grid, st);
    else if (q_dtype == TQ_DTYPE_BF16) r = launch_score_q<__nv_bfloat16>(A, o->bounds_dtype, grid, st);
    else r = launch_score_q<__half>(A, o->bounds_dtype, grid, st);
    if (r != TQ_OK) return r;
  }
  page_pick_kernel<<<(unsigned)(B * Hkv), kSelThreads, 0, st>>>(A);
  count_launch();
  return check_launch("page_pick_kernel");
}

}  // namespace tq
