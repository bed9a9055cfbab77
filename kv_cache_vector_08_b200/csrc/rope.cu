// Rotary positions of queries and keys, ahead of tq_quantize_kv and the attention calls.
//
// Pair i of a head turns by the angle a = pos * freq_i:
//   y1 = f (x1 cos a - x2 sin a),   y2 = f (x2 cos a + x1 sin a)
// with (x1, x2) = (x[i], x[i + rot/2]) or, interleaved, (x[2i], x[2i+1]); channels from rot
// on are copied.  The transposed rotation (the gradient, and for f = 1 the inverse) turns by -a.
//
// The angle is formed in 64 bits as a number of turns, pos * (freq / 2 pi), of which only the
// fraction is kept, in 32 bits: for frequencies up to 1 the angle is good to 1e-7 at positions up
// to 2^25, where that rounding is all of it, to 5e-7 at 2^31 and from there on in proportion to the
// position (the 64-bit product's own rounding; largest errors of 100,000 random angles against 60
// digits).  A 32-bit product would be off by whole turns.  Its sine and cosine are taken once per
// token and pair of a block, in shared memory, and serve all heads of both tensors.
//
// Bound: HBM (every element is read and written once).  A thread moves one vector of each
// half of the pairs (half layout) or two adjacent ones (interleaved) at a time; queries and
// keys go in one launch, since for a decode step the launch is the cost.  32,768 tokens of 32 + 8 heads
// of 128 channels (bf16, 671 MB): 111 us, 6.0 TB/s, 0.92 of a copy's rate; 64 tokens: 2.3 us.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "elem.cuh"
#include "kernels.cuh"

namespace tq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRowBytes = 16 * 1024;   // of whole rows in a block's shared memory
constexpr int64_t kRopeMaxRow = 1 << 19;   // elements of one token over both tensors

// n / d for n d < 2^40, n < 2^20 by one multiplication
struct Div {
  uint64_t m;
  int d;
  Div(int d_ = 1) : m(((1ull << 40) + d_ - 1) / d_), d(d_) {}
  __device__ __forceinline__ int quot(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> 40); }
};

struct RopeSide {
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh;   // strides in elements: token, head
};

struct RopeArgs {
  RopeSide s[2];
  int heads0;               // heads of the first tensor
  int64_t n;
  int rot, D;
  int tb;                   // tokens per block
  int per_block;            // units of a block (tb * heads * units)
  int chunk;                // units per grid.y slice
  Div per_tok, per_head;    // units of a token, units of a head (whole rows: rows of a token, pieces of a row)
  Div per_row;              // pairs of a row
  int rot_units;            // units of a head that rotate (the others copy)
  const double* freq;
  const void* pos;
  int pos64;
  float factor, sign;
};

// (written out, so that every kernel rounds alike)
__device__ __forceinline__ void turn_pair(float x1, float x2, float2 w, float& y1, float& y2) {
  y1 = fmaf(x1, w.x, -(x2 * w.y));
  y2 = fmaf(x2, w.x, x1 * w.y);
}

// Cosines and sines, times the factor, of tokens t0 .. t0 + ntok - 1.  Units of eight pairs read them two at a time
// from an order in which pairs 2 m and 2 m + 1 of all units are neighbours; in the order of the pairs the lanes'
// reads met in four banks (16,384 tokens of 40 heads, bf16: 66 us instead of 61).  Units of four (32-bit types) gain
// nothing from it (5,001 tokens of 15 heads of 96, 40 turning: 12.6 us, 12.0 in the plain order).
template <int V>
__device__ __forceinline__ int angle_slot(int np, int k, int j) {
  return V < 8 ? V * k + j : ((j >> 1) * (np / V) + k) * 2 + (j & 1);
}
template <int V>
__device__ __forceinline__ void form_angles(const RopeArgs& A, int64_t t0, int ntok, float2* cs) {
  const int np = A.rot / 2;
  for (int e = threadIdx.x; e < ntok * np; e += kRopeThreads) {
    const int t = e / np, i = e - t * np;
    const double pos = A.pos64 ? (double)static_cast<const int64_t*>(A.pos)[t0 + t]
                               : (double)static_cast<const int32_t*>(A.pos)[t0 + t];
    const double turns = pos * (A.freq[i] * 0.15915494309189533577);
    float si, co;
    sincospif((float)(2.0 * (turns - rint(turns))), &si, &co);
    cs[t * np + angle_slot<V>(np, i / V, i % V)] = make_float2(co * A.factor, si * A.factor * A.sign);
  }
}

template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_kernel(const __grid_constant__ RopeArgs A) {
  extern __shared__ __align__(16) float2 s_cs[];   // [tb][rot / 2] (cos, sin), times the factor
  using VT = Vec<T, V>;
  const int64_t t0 = (int64_t)blockIdx.x * A.tb;
  const int ntok = (int)(A.n - t0 < A.tb ? A.n - t0 : A.tb), np = A.rot / 2;
  const int u0 = blockIdx.y * A.chunk, u1 = min(u0 + A.chunk, ntok * A.per_tok.d);
  // One unit: where it lies, what it holds.
  struct Unit {
    T* o;
    int t, k;                      // token of the block, unit of the head
    VT a, b;
  };
  auto fetch = [&](int u, Unit& x) {
    x.t = A.per_tok.quot(u);
    const int r = u - x.t * A.per_tok.d;
    int h = A.per_head.quot(r);
    x.k = r - h * A.per_head.d;
    const bool second = h >= A.heads0;
    h -= second ? A.heads0 : 0;
    // (selected field by field: an indexed parameter struct would be copied to local memory)
    const T* p = static_cast<const T*>(second ? A.s[1].x : A.s[0].x) +
                 (t0 + x.t) * (second ? A.s[1].xt : A.s[0].xt) + h * (second ? A.s[1].xh : A.s[0].xh);
    x.o = static_cast<T*>(second ? A.s[1].out : A.s[0].out) +
          (t0 + x.t) * (second ? A.s[1].ot : A.s[0].ot) + h * (second ? A.s[1].oh : A.s[0].oh);
    if (x.k >= A.rot_units) {
      x.a = *reinterpret_cast<const VT*>(p + A.rot + (x.k - A.rot_units) * V);
    } else {
      // V pairs: vectors of both halves, or (interleaved) two adjacent ones
      x.a = *reinterpret_cast<const VT*>(p + (INTER ? 2 * V : V) * x.k);
      x.b = *reinterpret_cast<const VT*>(p + (INTER ? 2 * V * x.k + V : V * x.k + np));
    }
  };
  auto turn = [&](Unit& x) {
    if (x.k >= A.rot_units) {
      *reinterpret_cast<VT*>(x.o + A.rot + (x.k - A.rot_units) * V) = x.a;
      return;
    }
    const float2* cs = s_cs + x.t * np;
    float4 two;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (V >= 8 && j % 2 == 0) two = *reinterpret_cast<const float4*>(cs + angle_slot<V>(np, x.k, j));
      const float2 w = V < 8 ? cs[angle_slot<V>(np, x.k, j)] : j % 2 ? make_float2(two.z, two.w) : make_float2(two.x, two.y);
      // pair j: elements j of the vectors, or (interleaved) elements 2 j and 2 j + 1 of both in a row
      T& y = INTER ? (2 * j < V ? x.a.v[2 * j % V] : x.b.v[2 * j % V]) : x.a.v[j];
      T& z = INTER ? (2 * j + 1 < V ? x.a.v[(2 * j + 1) % V] : x.b.v[(2 * j + 1) % V]) : x.b.v[j];
      float y1, y2;
      turn_pair(to_f<T>(y), to_f<T>(z), w, y1, y2);
      y = from_f<T>(y1);
      z = from_f<T>(y2);
    }
    *reinterpret_cast<VT*>(x.o + (INTER ? 2 * V : V) * x.k) = x.a;
    *reinterpret_cast<VT*>(x.o + (INTER ? 2 * V * x.k + V : V * x.k + np)) = x.b;
  };
  // The thread's first unit is on its way while the angles are formed.  (One unit at a time and many
  // warps: four units a thread need 126 registers, and with 16 warps an SM the 32K prompt took 218 us; two
  // units, 32 warps: 134 us; one, 32 or 40 warps: 127 and 125 us; 48 spill: 127 us; later steps took the 40 to 111.)
  Unit x;
  int u = u0 + threadIdx.x;
  if (u < u1) fetch(u, x);
  form_angles<V>(A, t0, ntok, s_cs);
  __syncthreads();
  while (u < u1) {
    turn(x);
    u += kRopeThreads;
    if (u < u1) fetch(u, x);
  }
}

// The same where the halves are no multiples of 16 bytes but whole rows are (a row: one head of one token): rows
// come to shared memory 16 bytes at a time, turn there pair by pair, and go out 16 bytes at a time.
// 16,384 tokens of 32 + 8 heads of 128 channels, 50 of them turning (bf16, 336 MB): 77 us, 0.67 of a copy's rate;
// the kernel above with its narrow pieces takes 333 us (interleaved 215 us, 52 channels 177 us).  Rows whose halves
// are multiples of 16 bytes stay with the kernel above: 61 us where this one takes 101 us.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeArgs A) {
  extern __shared__ __align__(16) uint8_t s_rows[];   // [chunk][D], then [tb][rot / 2] (cos, sin)
  T* rows = reinterpret_cast<T*>(s_rows);
  float2* s_cs = reinterpret_cast<float2*>(s_rows + (size_t)A.chunk * A.D * sizeof(T));
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t t0 = (int64_t)blockIdx.x * A.tb;
  const int ntok = (int)(A.n - t0 < A.tb ? A.n - t0 : A.tb), np = A.rot / 2;
  const int r0 = blockIdx.y * A.chunk, nrow = min(A.chunk, ntok * A.per_tok.d - r0);    // rows of the block's tokens
  // element 16-byte piece e of the block's rows is at
  auto piece = [&](int e, bool out) -> uint8_t* {
    const int r = A.per_head.quot(e), c = e - r * A.per_head.d, t = A.per_tok.quot(r0 + r);
    int h = r0 + r - t * A.per_tok.d;
    const bool second = h >= A.heads0;
    h -= second ? A.heads0 : 0;
    const int64_t at = out ? (t0 + t) * (second ? A.s[1].ot : A.s[0].ot) + h * (second ? A.s[1].oh : A.s[0].oh)
                           : (t0 + t) * (second ? A.s[1].xt : A.s[0].xt) + h * (second ? A.s[1].xh : A.s[0].xh);
    const void* base = out ? (second ? A.s[1].out : A.s[0].out) : (second ? A.s[1].x : A.s[0].x);
    return const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + (at + c * V) * (int64_t)sizeof(T);
  };
  for (int e = threadIdx.x; e < nrow * A.per_head.d; e += kRopeThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(s_rows + (size_t)e * 16)),
                 "l"(piece(e, false)) : "memory");
  form_angles<1>(A, t0, ntok, s_cs);
  asm volatile("cp.async.wait_all;\n" ::: "memory");
  __syncthreads();
  for (int e = threadIdx.x; e < nrow * np; e += kRopeThreads) {
    const int r = A.per_row.quot(e), i = e - r * np;
    T* x = rows + r * A.D + (INTER ? 2 * i : i);
    T* z = x + (INTER ? 1 : np);
    float y1, y2;
    turn_pair(to_f<T>(*x), to_f<T>(*z), s_cs[A.per_tok.quot(r0 + r) * np + i], y1, y2);
    *x = from_f<T>(y1);
    *z = from_f<T>(y2);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nrow * A.per_head.d; e += kRopeThreads)
    *reinterpret_cast<uint4*>(piece(e, true)) = *reinterpret_cast<const uint4*>(s_rows + (size_t)e * 16);
}

template <typename T>
int launch_rows(RopeArgs A, int heads, bool inter, int sms, cudaStream_t st) {
  A.per_head = Div(A.D * (int)sizeof(T) / 16);
  A.per_tok = Div(heads);
  A.per_row = Div(A.rot / 2);
  const int most = std::max(1, kRopeRowBytes / (A.D * (int)sizeof(T)));       // rows a block
  int64_t tb = std::max<int64_t>(1, most / heads);
  tb = std::max<int64_t>(1, std::min<int64_t>(tb, A.n / (4 * sms)));
  tb = std::min<int64_t>(tb, std::max(1, 16 * 1024 / (A.rot / 2 * (int)sizeof(float2))));
  A.tb = (int)tb;
  const int64_t blocks = (A.n + tb - 1) / tb;
  const int rows = A.tb * heads;
  int64_t slices = (rows + most - 1) / most;
  if (blocks * slices < 2 * sms) slices = std::min<int64_t>((2 * sms + blocks - 1) / blocks, rows);
  A.chunk = (int)((rows + slices - 1) / slices);
  slices = (rows + A.chunk - 1) / A.chunk;
  const dim3 grid((unsigned)blocks, (unsigned)slices);
  const size_t sm = (size_t)A.chunk * A.D * sizeof(T) + (size_t)A.tb * (A.rot / 2) * sizeof(float2);
  if (inter) rope_rows_kernel<T, true><<<grid, kRopeThreads, sm, st>>>(A);
  else rope_rows_kernel<T, false><<<grid, kRopeThreads, sm, st>>>(A);
  count_launch();
  return check_launch("rope_rows_kernel");
}

template <typename T, int V>
int launch_v(RopeArgs A, int heads, bool inter, int sms, cudaStream_t st) {
  A.rot_units = A.rot / 2 / V;
  const int per_head = A.rot_units + (A.D - A.rot) / V;
  A.per_head = Div(per_head);
  A.per_tok = Div(per_head * heads);
  // A block takes about eight units a thread (the 32K prompt with cold caches: two 152 us, four 121, eight
  // and twelve 119): whole tokens (their sines are shared by the heads), or, when the tokens are too few for the device, slices of one token's heads.
  const int want = 8 * kRopeThreads;
  int64_t tb = std::max<int64_t>(1, want / A.per_tok.d);
  tb = std::max<int64_t>(1, std::min<int64_t>(tb, A.n / (4 * sms)));
  tb = std::min<int64_t>(tb, std::max(1, 24 * 1024 / std::max(1, A.rot / 2 * (int)sizeof(float2))));
  A.tb = (int)tb;
  A.per_block = A.tb * A.per_tok.d;
  const int64_t blocks = (A.n + tb - 1) / tb;
  int slices = 1;
  if (blocks < 2 * sms) slices = (int)std::min<int64_t>((2 * sms + blocks - 1) / blocks, (A.per_block + kRopeThreads - 1) / kRopeThreads);
  A.chunk = (A.per_block + slices - 1) / slices;
  slices = (A.per_block + A.chunk - 1) / A.chunk;
  const dim3 grid((unsigned)blocks, (unsigned)slices);
  const size_t sm = (size_t)A.tb * (A.rot / 2) * sizeof(float2);
  if (inter) rope_kernel<T, V, true><<<grid, kRopeThreads, sm, st>>>(A);
  else rope_kernel<T, V, false><<<grid, kRopeThreads, sm, st>>>(A);
  count_launch();
  return check_launch("rope_kernel");
}

template <typename T>
int launch_t(const RopeArgs& A, int heads, bool inter, int vec, bool rows, int sms, cudaStream_t st) {
  if (rows) return launch_rows<T>(A, heads, inter, sms, st);
  if constexpr (sizeof(T) == 2)
    if (vec >= 8) return launch_v<T, 8>(A, heads, inter, sms, st);
  if (vec >= 4) return launch_v<T, 4>(A, heads, inter, sms, st);
  if (vec >= 2) return launch_v<T, 2>(A, heads, inter, sms, st);
  return launch_v<T, 1>(A, heads, inter, sms, st);
}

}  // namespace

int launch_rope(const tq_rope_tensor* t, int nt, int dtype, int64_t n, int D, int rot, const double* freq,
                const void* pos, int pos_bits, double factor, int flags, cudaStream_t st) {
  const int es = dtype == TQ_DTYPE_F32 ? 4 : 2;
  const bool inter = (flags & TQ_ROPE_INTERLEAVED) != 0;
  RopeArgs A{};
  int heads = 0;
  // widest vector that divides the rotating halves and the copied rest, and that
  // every pointer and stride is aligned to
  int vec = 16 / es;
  bool rows = D % vec == 0;               // whole rows in pieces of 16 bytes
  const int full = vec;
  auto fit = [&](int64_t elems) { while (vec > 1 && elems % vec != 0) vec /= 2; };
  auto fit_ptr = [&](const void* p) { while (vec > 1 && reinterpret_cast<uintptr_t>(p) % ((size_t)vec * es) != 0) vec /= 2; };
  fit(rot / 2);
  fit(D - rot);
  int at = 0;
  for (int i = 0; i < nt; ++i) {
    if (t[i].heads == 0) continue;
    RopeSide& s = A.s[at++];
    s = RopeSide{t[i].x, t[i].out, t[i].x_token, t[i].x_head, t[i].out_token, t[i].out_head};
    if (at == 1) A.heads0 = t[i].heads;
    heads += t[i].heads;
    rows = rows && reinterpret_cast<uintptr_t>(s.x) % 16 == 0 && reinterpret_cast<uintptr_t>(s.out) % 16 == 0 &&
           (n <= 1 || (s.xt % full == 0 && s.ot % full == 0)) && (t[i].heads <= 1 || (s.xh % full == 0 && s.oh % full == 0));
    fit_ptr(s.x);
    fit_ptr(s.out);
    for (int64_t v : {s.xt, s.ot}) if (n > 1) fit(v);
    for (int64_t v : {s.xh, s.oh}) if (t[i].heads > 1) fit(v);
  }
  if (at == 0) return TQ_OK;
  rows = rows && vec < full;
  if ((int64_t)heads * D > kRopeMaxRow)
    return fail(TQ_ERR_UNSUPPORTED, "tq_rope: one token has more than 2^19 elements");
  A.n = n; A.rot = rot; A.D = D; A.freq = freq; A.pos = pos; A.pos64 = pos_bits == 64;
  A.factor = (float)factor;
  A.sign = (flags & TQ_ROPE_TRANSPOSE) ? -1.f : 1.f;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "tq_rope: device query");
  if (dtype == TQ_DTYPE_F32) return launch_t<float>(A, heads, inter, vec, rows, sms, st);
  if (dtype == TQ_DTYPE_BF16) return launch_t<__nv_bfloat16>(A, heads, inter, vec, rows, sms, st);
  return launch_t<__half>(A, heads, inter, vec, rows, sms, st);
}

// Frequencies of the usual long-context rules (host, 64 bits).
int rope_frequencies(int rot, double base, const tq_rope_scaling* s, double* freq, double* factor) {
  const int np = rot / 2;
  const double two_pi = 2.0 * M_PI;
  const int kind = s ? s->kind : TQ_ROPE_SCALE_NONE;
  if (kind == TQ_ROPE_SCALE_NTK) base *= std::pow(s->factor, rot > 2 ? (double)rot / (rot - 2) : 1.0);
  for (int i = 0; i < np; ++i) freq[i] = std::pow(base, -2.0 * i / rot);
  *factor = 1.0;
  if (kind == TQ_ROPE_SCALE_LINEAR) {
    for (int i = 0; i < np; ++i) freq[i] /= s->factor;
  } else if (kind == TQ_ROPE_SCALE_BANDS) {
    for (int i = 0; i < np; ++i) {
      const double turns = s->original_len * freq[i] / two_pi;
      const double w = std::min(1.0, std::max(0.0, (turns - s->low) / (s->high - s->low)));
      freq[i] *= w + (1.0 - w) / s->factor;
    }
  } else if (kind == TQ_ROPE_SCALE_YARN) {
    // pair index at which a frequency makes `turns` turns over the original length
    auto pair = [&](double turns) { return rot * std::log(s->original_len / (turns * two_pi)) / (2.0 * std::log(base)); };
    const double lo = std::max(std::floor(pair(s->high)), 0.0), hi = std::min(std::ceil(pair(s->low)), rot - 1.0);
    for (int i = 0; i < np; ++i) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      freq[i] = freq[i] / s->factor * ramp + freq[i] * (1.0 - ramp);
    }
    *factor = s->factor > 1.0 ? 0.1 * std::log(s->factor) + 1.0 : 1.0;
  }
  return TQ_OK;
}

}  // namespace tq
