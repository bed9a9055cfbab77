// Launchers of the libtq kernels (host side).
#pragma once

#include "common.cuh"

namespace tq {

// Returned by a kernel family's launcher when it does not cover the requested shape.
constexpr int kNotHandled = -1;

int launch_prepare_queries(const tq_ctx* ctx, const void* q, int q_dtype, int64_t nq, int64_t ld, float* out,
                           int64_t out_ld, cudaStream_t st);
void decode_geometry(int B, int Hkv, int64_t max_len, int* nsplit, int* chunk);
int decode_mma_ctas_per_sm();
struct DecodeWs {
  size_t qp, part, total;       // byte offsets of the regions and total size
  int nsplit, chunk;
  int64_t part_ld;              // floats per query row of the split partials (16-byte multiple)
};
DecodeWs decode_ws(int B, int Hq, int Hkv, int D, int G, int64_t max_len);
// How a caller that is not tq_decode_attention sees the call's heads: the output type, and, when
// each kv head is passed as a sequence of its own, the model's head counts (which the channel
// permutation goes by).
struct DecodeView {
  int out_dtype = TQ_DTYPE_F32;
  int perm_Hq = 0, perm_Hkv = 0;   // 0: the call's own
  // launch_decode_prep ran already, and the launch directly in front writes seq_lens and the table: the
  // decode kernel reads neither before its grid-dependency wait
  bool prepared = false;
};
size_t decode_workspace_bytes(int B, int Hq, int Hkv, int D, int ngroups, int64_t max_len, int qp_ld);
int launch_dequantize_tc(const tq_ctx* ctx, const tq_packed* src, const int64_t* slots, int64_t n, float* out,
                         int64_t ld, bool qjl, cudaStream_t st);
size_t quantize_gen_workspace(const tq_ctx* ctx, int64_t n);
int launch_quantize_gen(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const int32_t* cols,
                        const tq_packed* dst, const int64_t* slots, void* ws, size_t ws_bytes, cudaStream_t st);
bool quantize_tc_applies(const tq_ctx* ctx, int x_dtype, int64_t n, int64_t ld);
int launch_quantize_tc(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const tq_packed* dst,
                       const int64_t* slots, cudaStream_t st);
int launch_decode_mma(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* off, int G,
                      const int32_t* perm, const int32_t* table, int page, const void* q, int q_dtype,
                      const tq_packed* kc, const tq_packed* vc, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                      int64_t max_len, float scale, void* out, void* ws, cudaStream_t st,
                      const DecodeView& view = DecodeView());
int launch_decode_prep(const tq_ctx* const* kctx, const int* off, int G, const int32_t* perm, const void* q,
                       int q_dtype, int B, int Hq, int Hkv, int D, int64_t max_len, void* ws, const DecodeView& view,
                       cudaStream_t st);
bool decode_caches_supported(const tq_ctx* const* kctx, const tq_ctx* const* vctx, int G, const tq_packed* kc,
                             const tq_packed* vc);
size_t logits_mma_workspace(int64_t nq, int d);
int launch_logits_mma(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* keys, int64_t n, float* out,
                      void* ws, cudaStream_t st);
int launch_rope(const tq_rope_tensor* t, int nt, int dtype, int64_t n, int D, int rot, const double* freq,
                const void* pos, int pos_bits, double factor, int flags, cudaStream_t st);
int rope_frequencies(int rot, double base, const tq_rope_scaling* s, double* freq, double* factor);
int launch_page_bounds(const void* k, int64_t n, int dtype, int64_t k_token, int64_t k_head, const int32_t* cu_new,
                       const int32_t* start, int B, int Hkv, int D, int64_t max_new, const int32_t* table,
                       int page, int max_pages, void* bounds, int64_t npages, cudaStream_t st);
struct SparseWs {
  size_t key, vtable, vlen, decode, total;   // byte offsets of the regions and total size
};
SparseWs sparse_ws(int B, int Hq, int Hkv, int D, int G, int page, int max_pages, int select);
int launch_page_select(const void* q, int q_dtype, const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                       int64_t max_len, int64_t pool, const tq_sparse_opts* o, void* ws, const SparseWs& W,
                       cudaStream_t st);
size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int64_t max_len);
int launch_tree_attention(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* off, int G,
                          const int32_t* perm, const int32_t* table, int page, const void* q, int q_dtype,
                          const tq_packed* kc, const tq_packed* vc, const int32_t* seq_lens,
                          const int32_t* draft_lens, const uint64_t* mask, int B, int T, int Hq, int Hkv, int D,
                          int64_t max_len, float scale, void* out, void* ws, cudaStream_t st);
size_t search_tc_workspace(const tq_ctx* ctx, int64_t nq, int64_t N, int k);
int launch_search_tc(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* db, int64_t N, int k,
                     float* scores, int64_t* ids, void* ws, cudaStream_t st);
int launch_search_merge(float* cand_s, int64_t* cand_i, int64_t nq, int64_t ncand, int k, float* scores, int64_t* ids,
                        cudaStream_t st);

}  // namespace tq

namespace tq {
// Dispatchers: pick the fastest kernel family that supports the shape.
int launch_quantize(const tq_ctx* ctx, const void* x, int x_dtype, int64_t n, int64_t ld, const tq_packed* dst,
                    const int64_t* slots, void* ws, size_t ws_bytes, cudaStream_t st);
int launch_logits(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* keys, int64_t n, float* logits,
                  void* ws, cudaStream_t st);
int launch_decode(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* off, int G, const int32_t* perm,
                  const int32_t* table, int page, const void* q, int q_dtype, const tq_packed* kc,
                  const tq_packed* vc, const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len,
                  float scale, float* out, void* ws, cudaStream_t st);
int check_decode_args(const tq_ctx* const* kctx, const tq_ctx* const* vctx, const int* group_off, int ngroups,
                      const void* q, int q_dtype, const tq_packed* kcache, const tq_packed* vcache,
                      const int32_t* seq_lens, int B, int Hq, int Hkv, int D, int64_t max_len, const void* out,
                      int page, bool any_dtype = false);
int launch_search(const tq_ctx* ctx, const float* q, int64_t nq, const tq_packed* db, int64_t N, int k,
                  float* scores, int64_t* ids, void* ws, cudaStream_t st);
}  // namespace tq
