// C ABI of the fp8attn library: argument checks, context and workspace
// handling, selector parsing, static-scale import/export and the launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "fp8attn.h"
#include "kernels.h"
#include "state.cuh"

using namespace fp8attn;

struct fp8attn_ctx {
  int layers;
  int device;
  GlobalState* gs;
  LayerState* ls;
  std::vector<uint8_t> has_static;
};

namespace {

std::atomic<uint64_t> g_launches{0};

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline bool layer_ok(const fp8attn_ctx* c, int layer) {
  return c && layer >= 0 && layer < c->layers;
}

fp8attn_status status_of_bits(uint32_t bits) {
  if (bits & kErrTimeout) return FP8ATTN_ERR_TIMEOUT;
  if (bits & kErrSeqlens) return FP8ATTN_ERR_SEQLENS;
  if (bits & kErrPages) return FP8ATTN_ERR_PAGES;
  if (bits & kErrNonfinite) return FP8ATTN_ERR_NONFINITE;
  return FP8ATTN_OK;
}

__global__ void set_static_kernel(LayerState* ls, float q, float k, float v) {
  if (threadIdx.x != 0) return;
  const float A[3] = {q, k, v};
  for (int t = 0; t < 3; ++t) {
    ls->static_bound[t] = A[t];
    scales_from_bound(A[t], &ls->static_qs[t], &ls->static_ds[t]);
  }
}

// shared shape checks of the attention entry points
fp8attn_status check_attention(const void* q, const void* k, const void* v,
                               const int32_t* cu, int batch, int max_seqlen,
                               int64_t total_tokens, int num_heads, int head_dim, void* out) {
  if (batch < 1 || max_seqlen < 0 || num_heads < 1 || total_tokens < 0) return FP8ATTN_ERR_INVALID;
  if (head_dim != kHeadDim) return FP8ATTN_ERR_UNSUPPORTED;
  if (!cu) return FP8ATTN_ERR_INVALID;
  if (total_tokens > static_cast<int64_t>(batch) * max_seqlen) return FP8ATTN_ERR_INVALID;
  if (total_tokens > 0x7FFFFFFFLL) return FP8ATTN_ERR_UNSUPPORTED;
  if (total_tokens == 0) return FP8ATTN_OK;
  if (!q || !k || !v || !out) return FP8ATTN_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
    return FP8ATTN_ERR_INVALID;
  return FP8ATTN_OK;
}

fp8attn_status run_attention(const void* q, const void* k, const void* v, const int32_t* cu,
                             int batch, int max_seqlen, int64_t total_tokens, int num_heads,
                             int head_dim, const float* descale, float softmax_scale, void* out,
                             int32_t* err, void* stream, int bf16, int p_rule,
                             int schedule) {
  if (p_rule != FP8ATTN_P_LINEAR_LOG && p_rule != FP8ATTN_P_EXP2) return FP8ATTN_ERR_INVALID;
  if (schedule != FP8ATTN_SCHED_AUTO && schedule != FP8ATTN_SCHED_WHOLE &&
      schedule != FP8ATTN_SCHED_SPLIT)
    return FP8ATTN_ERR_INVALID;
  fp8attn_status st = check_attention(q, k, v, cu, batch, max_seqlen, total_tokens, num_heads,
                                      head_dim, out);
  if (st != FP8ATTN_OK || total_tokens == 0) return st;
  if (!bf16 && !descale) return FP8ATTN_ERR_INVALID;
  if (!(softmax_scale >= 0.0f) || std::isinf(softmax_scale)) return FP8ATTN_ERR_INVALID;
  AttnLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu = cu;
  a.batch = batch;
  a.heads = num_heads;
  a.max_seqlen = max_seqlen;
  a.descale = descale;
  a.softmax_scale = softmax_scale == 0.0f ? 1.0f / std::sqrt(static_cast<float>(head_dim))
                                          : softmax_scale;
  a.out = out;
  a.err = err;
  a.bf16 = bf16;
  a.p_rule = p_rule == FP8ATTN_P_EXP2 ? kPRuleExp2 : kPRuleLinearLog;
  a.schedule = schedule == FP8ATTN_SCHED_WHOLE   ? kSchedWhole
               : schedule == FP8ATTN_SCHED_SPLIT ? kSchedSplit
                                                 : kSchedAuto;
  const cudaError_t e = launch_attention(a, total_tokens, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

// log2 of a page size the paged cache supports (8 to 1024 slots), or -1
int page_log2_of(int page_size) {
  for (int l = 3; l <= 10; ++l)
    if (page_size == 1 << l) return l;
  return -1;
}

// Shared checks of a paged cache.  The strides of a dimension of size one do
// not matter; they are replaced by ones that the kernels accept.
fp8attn_status check_cache(const void* k, const void* v, int64_t page_stride, int64_t slot_stride,
                           int64_t head_stride, int num_pages, int page_size, int heads,
                           int head_dim, bool fp8, PagedCache* out) {
  if (num_pages < 1 || page_size < 1 || heads < 1) return FP8ATTN_ERR_INVALID;
  if (head_dim != kHeadDim || page_log2_of(page_size) < 0) return FP8ATTN_ERR_UNSUPPORTED;
  if (!k || !v) return FP8ATTN_ERR_INVALID;
  if (num_pages == 1) page_stride = kHeadDim;
  if (heads == 1) head_stride = kHeadDim;
  const int64_t unit = fp8 ? 16 : 8;   // elements of 16 bytes
  for (int64_t s : {page_stride, slot_stride, head_stride})
    if (s < kHeadDim || s % unit || s >= int64_t{1} << 38) return FP8ATTN_ERR_UNSUPPORTED;
  if (!aligned(k, 16) || !aligned(v, 16)) return FP8ATTN_ERR_UNSUPPORTED;
  out->k = const_cast<void*>(k);
  out->v = const_cast<void*>(v);
  out->page_stride = page_stride;
  out->slot_stride = slot_stride;
  out->head_stride = head_stride;
  out->num_pages = num_pages;
  out->page_log2 = page_log2_of(page_size);
  out->heads = heads;
  out->fp8 = fp8;
  return FP8ATTN_OK;
}

// (`fp8` says what the cache holds; a scale does not, since a missing one must
// not turn an E4M3 cache into a bf16 one of twice the bytes)
fp8attn_status run_kv_write(const void* k, const void* v, int64_t tok_stride, int64_t head_stride,
                            const int64_t* d_slots, int64_t tokens, int num_kv_heads, int head_dim,
                            void* k_cache, void* v_cache, int64_t page_stride, int64_t slot_stride,
                            int64_t cache_head_stride, int num_pages, int page_size, bool fp8,
                            const float* qs, int32_t* d_error, void* stream) {
  if (tokens < 0) return FP8ATTN_ERR_INVALID;
  KvWriteLaunch p;
  const fp8attn_status st =
      check_cache(k_cache, v_cache, page_stride, slot_stride, cache_head_stride, num_pages,
                  page_size, num_kv_heads, head_dim, fp8, &p.cache);
  if (st != FP8ATTN_OK || tokens == 0) return st;
  if (!k || !v || !d_slots) return FP8ATTN_ERR_INVALID;
  if (tok_stride <= 0 || head_stride <= 0 || (tok_stride % 8) || (head_stride % 8) ||
      !aligned(k, 16) || !aligned(v, 16) || !aligned(d_slots, 8) ||
      tokens > 0x7FFFFFFFLL / num_kv_heads)
    return FP8ATTN_ERR_UNSUPPORTED;
  p.k = k;
  p.v = v;
  p.tok_stride = tok_stride;
  p.head_stride = head_stride;
  p.slots = d_slots;
  p.tokens = tokens;
  p.qs = qs;
  p.err = d_error;
  if (launch_kv_write(p, as_stream(stream)) != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status run_kv_tree(const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                           const void* k_cache, const void* v_cache, int64_t page_stride,
                           int64_t slot_stride, int64_t cache_head_stride, int num_pages,
                           int page_size, const int32_t* d_block_tables, int64_t table_stride,
                           int table_width, const int32_t* d_seq_lens, const int32_t* d_cu_q,
                           int rows, int max_q_len, int max_seqlen, int64_t total_q, int num_heads,
                           int num_kv_heads, int head_dim, bool fp8, const float* descale,
                           const int64_t* d_tree_mask, int mask_words, float softmax_scale,
                           void* out, void* workspace, size_t workspace_bytes, int32_t* d_error,
                           void* stream) {
  if (rows < 0 || max_q_len < 0 || max_seqlen < 0 || total_q < 0 || num_heads < 1 ||
      num_kv_heads < 1 || num_heads % num_kv_heads || table_width < 1 ||
      (d_tree_mask && mask_words < 1))
    return FP8ATTN_ERR_INVALID;
  if (!(softmax_scale >= 0.0f) || std::isinf(softmax_scale)) return FP8ATTN_ERR_INVALID;
  KvTreeLaunch p;
  const fp8attn_status st =
      check_cache(k_cache, v_cache, page_stride, slot_stride, cache_head_stride, num_pages,
                  page_size, num_kv_heads, head_dim, fp8, &p.cache);
  if (st != FP8ATTN_OK) return st;
  if (rows > kMaxTreeRows) return FP8ATTN_ERR_UNSUPPORTED;
  if (rows == 0 || total_q == 0) return FP8ATTN_OK;
  if (rows > 1 && table_stride < table_width) return FP8ATTN_ERR_INVALID;
  if (!q || !out || !d_block_tables || !d_seq_lens || !d_cu_q) return FP8ATTN_ERR_INVALID;
  if (q_tok_stride <= 0 || q_head_stride <= 0 || (q_tok_stride % 8) || (q_head_stride % 8) ||
      !aligned(q, 16) || !aligned(out, 16) || !aligned(d_tree_mask, 8) ||
      total_q > 0x7FFFFFFFLL / num_heads ||
      (num_heads / num_kv_heads) > 1024)
    return FP8ATTN_ERR_UNSUPPORTED;
  // no request has more queries than there are, nor tokens than its table holds
  if (max_q_len > total_q) max_q_len = static_cast<int>(total_q);
  const int64_t held = static_cast<int64_t>(table_width) * page_size;
  if (max_seqlen > held) max_seqlen = static_cast<int>(held);
  // the kernels hold query rows, positions and their ends (a tile further) in
  // 32 bits, and divide query rows by the group in 32 bits
  const int64_t group = num_heads / num_kv_heads;
  if ((max_q_len * group + 128) * group > 0xFFFFFFFFLL || max_q_len * group > 0x7FFFFF00LL ||
      max_seqlen > 0x7FFFFF00LL ||
      kv_tree_max_items(rows, max_q_len, max_seqlen, num_heads, num_kv_heads) > 0x7FFFFFFFLL)
    return FP8ATTN_ERR_UNSUPPORTED;
  const size_t need =
      max_q_len && max_seqlen
          ? kv_tree_workspace_bytes(rows, max_q_len, max_seqlen, num_heads, num_kv_heads)
          : 0;
  if (need > workspace_bytes || (need && !workspace)) return FP8ATTN_ERR_INVALID;
  if (!aligned(workspace, 16)) return FP8ATTN_ERR_UNSUPPORTED;
  p.q = q;
  p.q_tok_stride = q_tok_stride;
  p.q_head_stride = q_head_stride;
  p.tables = d_block_tables;
  p.table_stride = table_stride;
  p.width = table_width;
  p.seq = d_seq_lens;
  p.cu = d_cu_q;
  p.rows = rows;
  p.max_q = max_q_len;
  p.max_seqlen = max_seqlen;
  p.total_q = total_q;
  p.heads = num_heads;
  p.descale = descale;
  p.mask = d_tree_mask;
  p.mask_words = mask_words;
  p.softmax_scale = softmax_scale == 0.0f ? 1.0f / std::sqrt(static_cast<float>(head_dim))
                                          : softmax_scale;
  p.out = out;
  p.workspace = workspace;
  p.err = d_error;
  if (launch_kv_tree(p, as_stream(stream)) != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

}  // namespace

void fp8attn::note_launch() { g_launches.fetch_add(1); }

extern "C" {

const char* fp8attn_status_string(int status) {
  switch (status) {
    case FP8ATTN_OK: return "ok";
    case FP8ATTN_ERR_INVALID: return "invalid argument";
    case FP8ATTN_ERR_CUDA: return "CUDA error";
    case FP8ATTN_ERR_TIMEOUT: return "device wait timed out";
    case FP8ATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case FP8ATTN_ERR_NONFINITE: return "non-finite amax";
    case FP8ATTN_ERR_SEQLENS: return "inconsistent cu_seqlens";
    case FP8ATTN_ERR_PAGES: return "page outside the cache, or too few free pages";
    default: return "unknown status";
  }
}

int fp8attn_ring_length(void) { return kRing; }

size_t fp8attn_workspace_bytes(int num_layers) {
  return num_layers < 1 ? 0 : workspace_bytes_for(num_layers);
}

fp8attn_status fp8attn_create(int num_layers, void* d_workspace, size_t workspace_bytes,
                              void* stream, fp8attn_ctx** out) {
  if (!out) return FP8ATTN_ERR_INVALID;
  *out = nullptr;
  if (num_layers < 1 || !d_workspace || !aligned(d_workspace, 256) ||
      workspace_bytes < workspace_bytes_for(num_layers))
    return FP8ATTN_ERR_INVALID;
  fp8attn_ctx* c = new (std::nothrow) fp8attn_ctx;
  if (!c) return FP8ATTN_ERR_INVALID;
  c->layers = num_layers;
  c->gs = static_cast<GlobalState*>(d_workspace);
  c->ls = reinterpret_cast<LayerState*>(static_cast<char*>(d_workspace) + sizeof(GlobalState));
  c->has_static.assign(num_layers, 0);
  if (cudaGetDevice(&c->device) != cudaSuccess ||
      cudaMemsetAsync(d_workspace, 0, workspace_bytes_for(num_layers), as_stream(stream)) !=
          cudaSuccess) {
    delete c;
    return FP8ATTN_ERR_CUDA;
  }
  // empty rings: unit scales until the first pass
  std::vector<LayerState> init(num_layers);
  std::memset(init.data(), 0, sizeof(LayerState) * num_layers);
  for (auto& l : init)
    for (int t = 0; t < 3; ++t) l.qs[t] = l.ds[t] = l.static_qs[t] = l.static_ds[t] = 1.0f;
  if (cudaMemcpyAsync(c->ls, init.data(), sizeof(LayerState) * num_layers,
                      cudaMemcpyHostToDevice, as_stream(stream)) != cudaSuccess ||
      cudaStreamSynchronize(as_stream(stream)) != cudaSuccess) {
    delete c;
    return FP8ATTN_ERR_CUDA;
  }
  *out = c;
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_destroy(fp8attn_ctx* ctx) {
  if (!ctx) return FP8ATTN_ERR_INVALID;
  delete ctx;
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_quantize_qkv(fp8attn_ctx* ctx, int layer, int mode, const void* q,
                                    const void* k, const void* v, int64_t tok_stride,
                                    int64_t head_stride, const int32_t* d_src_seq_start,
                                    const int32_t* d_cu_seqlens, int batch, int max_seqlen,
                                    int64_t total_tokens, int num_heads, int head_dim, void* q8,
                                    void* k8, void* v8, void* stream) {
  if (!layer_ok(ctx, layer)) return FP8ATTN_ERR_INVALID;
  if (mode != FP8ATTN_DYNAMIC && mode != FP8ATTN_STATIC && mode != FP8ATTN_RING)
    return FP8ATTN_ERR_INVALID;
  if (mode == FP8ATTN_STATIC && !ctx->has_static[layer]) return FP8ATTN_ERR_INVALID;
  if (batch < 1 || max_seqlen < 0 || num_heads < 1 || total_tokens < 0 || !d_cu_seqlens)
    return FP8ATTN_ERR_INVALID;
  if (head_dim != kHeadDim) return FP8ATTN_ERR_UNSUPPORTED;
  if (total_tokens > static_cast<int64_t>(batch) * max_seqlen) return FP8ATTN_ERR_INVALID;
  if (!q || !k || !v || !q8 || !k8 || !v8) return FP8ATTN_ERR_INVALID;
  if (tok_stride <= 0 || head_stride <= 0 || (tok_stride % 8) || (head_stride % 8))
    return FP8ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q8, 16) ||
      !aligned(k8, 16) || !aligned(v8, 16))
    return FP8ATTN_ERR_UNSUPPORTED;
  QuantLaunch L;
  L.src[0] = q;
  L.src[1] = k;
  L.src[2] = v;
  L.dst[0] = q8;
  L.dst[1] = k8;
  L.dst[2] = v8;
  L.tok_stride = tok_stride;
  L.head_stride = head_stride;
  L.cu = d_cu_seqlens;
  L.src_seq_start = d_src_seq_start;
  L.batch = batch;
  L.heads = num_heads;
  L.max_seqlen = max_seqlen;
  L.total_tokens = total_tokens;
  L.kind = mode == FP8ATTN_DYNAMIC ? kQuantDynamic : mode == FP8ATTN_RING ? kQuantRing
                                                                           : kQuantStatic;
  L.amax_out = nullptr;
  L.gs = ctx->gs;
  L.ls = ctx->ls + layer;
  const cudaError_t e = launch_quantize(L, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_quantize_qkv_grouped(fp8attn_ctx* ctx, int layer, int mode, const void* q,
                                            const void* k, const void* v, int64_t tok_stride,
                                            int64_t head_stride, const int32_t* d_src_seq_start,
                                            const int32_t* d_cu_seqlens, int batch,
                                            int max_seqlen, int64_t total_tokens, int num_heads,
                                            int head_dim, int groups, void* q8, void* k8,
                                            void* v8, void* stream) {
  if (mode != FP8ATTN_STATIC && mode != FP8ATTN_RING) return FP8ATTN_ERR_INVALID;
  if (groups < 1 || num_heads < 1 || num_heads % groups) return FP8ATTN_ERR_INVALID;
  if (!layer_ok(ctx, layer)) return FP8ATTN_ERR_INVALID;
  if (mode == FP8ATTN_STATIC && !ctx->has_static[layer]) return FP8ATTN_ERR_INVALID;
  if (batch < 1 || max_seqlen < 0 || total_tokens < 0 || !d_cu_seqlens)
    return FP8ATTN_ERR_INVALID;
  if (head_dim != kHeadDim) return FP8ATTN_ERR_UNSUPPORTED;
  if (total_tokens > static_cast<int64_t>(batch) * max_seqlen) return FP8ATTN_ERR_INVALID;
  if (!q || !k || !v || !q8 || !k8 || !v8) return FP8ATTN_ERR_INVALID;
  if (tok_stride <= 0 || head_stride <= 0 || (tok_stride % 8) || (head_stride % 8))
    return FP8ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q8, 16) ||
      !aligned(k8, 16) || !aligned(v8, 16))
    return FP8ATTN_ERR_UNSUPPORTED;
  QuantLaunch L;
  L.src[0] = q;
  L.src[1] = k;
  L.src[2] = v;
  L.dst[0] = q8;
  L.dst[1] = k8;
  L.dst[2] = v8;
  L.tok_stride = tok_stride;
  L.head_stride = head_stride;
  L.cu = d_cu_seqlens;
  L.src_seq_start = d_src_seq_start;
  L.batch = batch;
  L.heads = num_heads;
  L.max_seqlen = max_seqlen;
  L.total_tokens = total_tokens;
  L.kind = mode == FP8ATTN_RING ? kQuantRing : kQuantStatic;
  L.amax_out = nullptr;
  L.gs = ctx->gs;
  L.ls = ctx->ls + layer;
  L.dst_groups = groups;
  const cudaError_t e = launch_quantize(L, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_amax_qkv(fp8attn_ctx* ctx, const void* q, const void* k, const void* v,
                                int64_t tok_stride, int64_t head_stride,
                                const int32_t* d_src_seq_start, const int32_t* d_cu_seqlens,
                                int batch, int max_seqlen, int64_t total_tokens, int num_heads,
                                int head_dim, float* d_amax3, void* stream) {
  if (!ctx || !d_amax3 || !aligned(d_amax3, 4)) return FP8ATTN_ERR_INVALID;
  if (batch < 1 || max_seqlen < 0 || num_heads < 1 || total_tokens < 0 || !d_cu_seqlens)
    return FP8ATTN_ERR_INVALID;
  if (head_dim != kHeadDim) return FP8ATTN_ERR_UNSUPPORTED;
  if (total_tokens > static_cast<int64_t>(batch) * max_seqlen) return FP8ATTN_ERR_INVALID;
  if (!q || !k || !v) return FP8ATTN_ERR_INVALID;
  if (tok_stride <= 0 || head_stride <= 0 || (tok_stride % 8) || (head_stride % 8))
    return FP8ATTN_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16)) return FP8ATTN_ERR_UNSUPPORTED;
  QuantLaunch L;
  L.src[0] = q;
  L.src[1] = k;
  L.src[2] = v;
  L.dst[0] = L.dst[1] = L.dst[2] = nullptr;
  L.tok_stride = tok_stride;
  L.head_stride = head_stride;
  L.cu = d_cu_seqlens;
  L.src_seq_start = d_src_seq_start;
  L.batch = batch;
  L.heads = num_heads;
  L.max_seqlen = max_seqlen;
  L.total_tokens = total_tokens;
  L.kind = kQuantAmaxOnly;
  L.amax_out = d_amax3;
  L.gs = ctx->gs;
  L.ls = ctx->ls;
  const cudaError_t e = launch_quantize(L, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_amax_ring_update(fp8attn_ctx* ctx, int layer, const float* d_amax3,
                                        void* stream) {
  if (!layer_ok(ctx, layer) || !d_amax3) return FP8ATTN_ERR_INVALID;
  const cudaError_t e = launch_ring_update(ctx->ls + layer, ctx->gs, d_amax3, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_set_static_scales(fp8attn_ctx* ctx, int layer, float q, float k,
                                         float v, void* stream) {
  if (!layer_ok(ctx, layer)) return FP8ATTN_ERR_INVALID;
  for (float x : {q, k, v})
    if (!std::isfinite(x) || x < 0.0f) return FP8ATTN_ERR_INVALID;
  set_static_kernel<<<1, 32, 0, as_stream(stream)>>>(ctx->ls + layer, q, k, v);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  ctx->has_static[layer] = 1;
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_clear_static_scales(fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer)) return FP8ATTN_ERR_INVALID;
  ctx->has_static[layer] = 0;
  return FP8ATTN_OK;
}

int fp8attn_has_static_scales(const fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer)) return -1;
  return ctx->has_static[layer] ? 1 : 0;
}

fp8attn_status fp8attn_export_static_scales(fp8attn_ctx* ctx, float margin, float* h_out,
                                            void* stream) {
  if (!ctx || !h_out || !std::isfinite(margin) || margin <= 0.0f) return FP8ATTN_ERR_INVALID;
  std::vector<LayerState> host(ctx->layers);
  cudaError_t e = cudaMemcpyAsync(host.data(), ctx->ls, sizeof(LayerState) * ctx->layers,
                                  cudaMemcpyDeviceToHost, as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  for (int l = 0; l < ctx->layers; ++l)
    for (int t = 0; t < 3; ++t) {
      float A = 0.0f;
      for (uint32_t i = 0; i < host[l].count[t] && i < static_cast<uint32_t>(kRing); ++i)
        A = std::fmax(A, host[l].ring[t][i]);
      volatile float prod = A * margin;   // one fp32 multiply
      h_out[l * 3 + t] = prod;
    }
  return FP8ATTN_OK;
}

const float* fp8attn_descale_ptr(fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer)) return nullptr;
  return ctx->ls[layer].ds;
}

const float* fp8attn_quant_scale_ptr(fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer)) return nullptr;
  return ctx->ls[layer].qs;
}

fp8attn_status fp8attn_get_ring_state(fp8attn_ctx* ctx, int layer, float* h_slots,
                                      uint32_t* h_meta, void* stream) {
  if (!layer_ok(ctx, layer) || !h_slots || !h_meta) return FP8ATTN_ERR_INVALID;
  LayerState host;
  cudaError_t e = cudaMemcpyAsync(&host, ctx->ls + layer, sizeof(LayerState),
                                  cudaMemcpyDeviceToHost, as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  std::memcpy(h_slots, host.ring, sizeof(host.ring));
  for (int t = 0; t < 3; ++t) {
    h_meta[2 * t] = host.head[t];
    h_meta[2 * t + 1] = host.count[t];
  }
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_set_ring_state(fp8attn_ctx* ctx, int layer, const float* h_slots,
                                      const uint32_t* h_meta, void* stream) {
  if (!layer_ok(ctx, layer) || !h_slots || !h_meta) return FP8ATTN_ERR_INVALID;
  for (int t = 0; t < 3; ++t) {
    const uint32_t head = h_meta[2 * t], count = h_meta[2 * t + 1];
    if (count > static_cast<uint32_t>(kRing) || head >= static_cast<uint32_t>(kRing))
      return FP8ATTN_ERR_INVALID;
    if (count < static_cast<uint32_t>(kRing) && head != count) return FP8ATTN_ERR_INVALID;
    for (int i = 0; i < kRing; ++i)
      if (!std::isfinite(h_slots[t * kRing + i]) || h_slots[t * kRing + i] < 0.0f)
        return FP8ATTN_ERR_INVALID;
  }
  LayerState host;
  cudaError_t e = cudaMemcpyAsync(&host, ctx->ls + layer, sizeof(LayerState),
                                  cudaMemcpyDeviceToHost, as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  std::memcpy(host.ring, h_slots, sizeof(host.ring));
  for (int t = 0; t < 3; ++t) {
    host.head[t] = h_meta[2 * t];
    host.count[t] = h_meta[2 * t + 1];
  }
  e = cudaMemcpyAsync(ctx->ls + layer, &host, sizeof(LayerState), cudaMemcpyHostToDevice,
                      as_stream(stream));
  if (e == cudaSuccess) e = launch_rescale_from_ring(ctx->ls + layer, as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_get_scales(fp8attn_ctx* ctx, int layer, float* h_out6, void* stream) {
  if (!layer_ok(ctx, layer) || !h_out6) return FP8ATTN_ERR_INVALID;
  LayerState host;
  cudaError_t e = cudaMemcpyAsync(&host, ctx->ls + layer, sizeof(LayerState),
                                  cudaMemcpyDeviceToHost, as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  for (int t = 0; t < 3; ++t) {
    h_out6[t] = host.qs[t];
    h_out6[3 + t] = host.ds[t];
  }
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_varlen_fwd(const void* q8, const void* k8, const void* v8,
                                  const int32_t* d_cu_seqlens, int batch, int max_seqlen,
                                  int64_t total_tokens, int num_heads, int head_dim,
                                  const float* d_descale_qkv, float softmax_scale, void* out,
                                  int32_t* d_error, void* stream) {
  return run_attention(q8, k8, v8, d_cu_seqlens, batch, max_seqlen, total_tokens, num_heads,
                       head_dim, d_descale_qkv, softmax_scale, out, d_error, stream, 0,
                       FP8ATTN_P_LINEAR_LOG, FP8ATTN_SCHED_AUTO);
}

fp8attn_status fp8attn_varlen_fwd_rule(const void* q8, const void* k8, const void* v8,
                                       const int32_t* d_cu_seqlens, int batch, int max_seqlen,
                                       int64_t total_tokens, int num_heads, int head_dim,
                                       const float* d_descale_qkv, float softmax_scale,
                                       int p_rule, void* out, int32_t* d_error, void* stream) {
  return run_attention(q8, k8, v8, d_cu_seqlens, batch, max_seqlen, total_tokens, num_heads,
                       head_dim, d_descale_qkv, softmax_scale, out, d_error, stream, 0, p_rule,
                       FP8ATTN_SCHED_AUTO);
}

fp8attn_status fp8attn_varlen_fwd_sched(const void* q8, const void* k8, const void* v8,
                                        const int32_t* d_cu_seqlens, int batch, int max_seqlen,
                                        int64_t total_tokens, int num_heads, int head_dim,
                                        const float* d_descale_qkv, float softmax_scale,
                                        int p_rule, int schedule, void* out, int32_t* d_error,
                                        void* stream) {
  return run_attention(q8, k8, v8, d_cu_seqlens, batch, max_seqlen, total_tokens, num_heads,
                       head_dim, d_descale_qkv, softmax_scale, out, d_error, stream, 0, p_rule,
                       schedule);
}

fp8attn_status fp8attn_varlen_fwd_static(fp8attn_ctx* ctx, int layer, const void* q,
                                         const void* k, const void* v, int64_t tok_stride,
                                         int64_t head_stride, const int32_t* d_cu_seqlens,
                                         int batch, int max_seqlen, int64_t total_tokens,
                                         int num_heads, int head_dim, float softmax_scale,
                                         int p_rule, void* out, void* stream) {
  if (!layer_ok(ctx, layer) || !ctx->has_static[layer]) return FP8ATTN_ERR_INVALID;
  if (p_rule != FP8ATTN_P_LINEAR_LOG && p_rule != FP8ATTN_P_EXP2) return FP8ATTN_ERR_INVALID;
  fp8attn_status st = check_attention(q, k, v, d_cu_seqlens, batch, max_seqlen, total_tokens,
                                      num_heads, head_dim, out);
  if (st != FP8ATTN_OK || total_tokens == 0) return st;
  if (!(softmax_scale >= 0.0f) || std::isinf(softmax_scale)) return FP8ATTN_ERR_INVALID;
  // rows of heads of 128 channels, heads within a row, no overlap; strides in
  // 16-byte units (the TMA map's rule)
  if (tok_stride <= 0 || head_stride <= 0 || (tok_stride % 8) || (head_stride % 8) ||
      head_stride < head_dim || tok_stride < static_cast<int64_t>(num_heads) * head_stride)
    return FP8ATTN_ERR_UNSUPPORTED;
  LayerState* ls = ctx->ls + layer;
  AttnLaunch a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu = d_cu_seqlens;
  a.batch = batch;
  a.heads = num_heads;
  a.max_seqlen = max_seqlen;
  a.descale = ls->static_ds;
  a.softmax_scale = softmax_scale == 0.0f ? 1.0f / std::sqrt(static_cast<float>(head_dim))
                                          : softmax_scale;
  a.out = out;
  a.err = reinterpret_cast<int32_t*>(&ctx->gs->error);
  a.bf16 = 0;
  a.p_rule = p_rule == FP8ATTN_P_EXP2 ? kPRuleExp2 : kPRuleLinearLog;
  a.schedule = kSchedAuto;
  a.fused = 1;
  a.tok_stride = tok_stride;
  a.head_stride = head_stride;
  a.qscale = ls->static_qs;
  a.cur_qs = ls->qs;
  a.cur_ds = ls->ds;
  const cudaError_t e = launch_attention(a, total_tokens, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_selftest_qk_scores(const void* d_q8, const void* d_k8, int64_t tiles,
                                          float* d_scores, int32_t* d_error, void* stream) {
  if (!d_q8 || !d_k8 || !d_scores || tiles < 1 || tiles > 0x7FFFFFFF / 128)
    return FP8ATTN_ERR_INVALID;
  if (!aligned(d_q8, 16) || !aligned(d_k8, 16) || !aligned(d_scores, 16))
    return FP8ATTN_ERR_INVALID;
  if (launch_qk_scores_probe(d_q8, d_k8, tiles, d_scores, d_error, as_stream(stream)) !=
      cudaSuccess)
    return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_varlen_fwd_bf16(const void* q, const void* k, const void* v,
                                       const int32_t* d_cu_seqlens, int batch, int max_seqlen,
                                       int64_t total_tokens, int num_heads, int head_dim,
                                       float softmax_scale, void* out, int32_t* d_error,
                                       void* stream) {
  return run_attention(q, k, v, d_cu_seqlens, batch, max_seqlen, total_tokens, num_heads,
                       head_dim, nullptr, softmax_scale, out, d_error, stream, 1,
                       FP8ATTN_P_EXP2, FP8ATTN_SCHED_WHOLE);
}

fp8attn_status fp8attn_get_error(fp8attn_ctx* ctx, void* stream) {
  if (!ctx) return FP8ATTN_ERR_INVALID;
  GlobalState host;
  cudaError_t e = cudaMemcpyAsync(&host, ctx->gs, sizeof(GlobalState), cudaMemcpyDeviceToHost,
                                  as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  const fp8attn_status st = status_of_bits(host.error);
  if (host.error) {
    // clear the error; after a timeout also reset the reduction words
    if (host.error & kErrTimeout) {
      e = cudaMemsetAsync(ctx->gs, 0, sizeof(GlobalState), as_stream(stream));
    } else {
      e = cudaMemsetAsync(&ctx->gs->error, 0, sizeof(uint32_t), as_stream(stream));
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
    if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  }
  return st;
}

fp8attn_status fp8attn_read_error_word(int32_t* d_error, void* stream) {
  if (!d_error) return FP8ATTN_ERR_INVALID;
  int32_t bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, d_error, sizeof(int32_t), cudaMemcpyDeviceToHost,
                                  as_stream(stream));
  if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  if (e == cudaSuccess && bits) {
    e = cudaMemsetAsync(d_error, 0, sizeof(int32_t), as_stream(stream));
    if (e == cudaSuccess) e = cudaStreamSynchronize(as_stream(stream));
  }
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  return status_of_bits(static_cast<uint32_t>(bits));
}

fp8attn_status fp8attn_parse_selector(const char* text, int max_index, uint8_t* mask_out) {
  if (max_index < 0 || (max_index > 0 && !mask_out)) return FP8ATTN_ERR_INVALID;
  if (max_index > 0) std::memset(mask_out, 0, static_cast<size_t>(max_index));
  if (!text) return FP8ATTN_OK;
  std::vector<uint8_t> mask(static_cast<size_t>(max_index), 0);
  const char* s = text;
  auto skip_ws = [&]() { while (*s == ' ' || *s == '\t') ++s; };
  auto read_int = [&](long* v) {
    if (*s < '0' || *s > '9') return false;
    long x = 0;
    while (*s >= '0' && *s <= '9') {
      x = x * 10 + (*s - '0');
      if (x > 1000000000L) return false;
      ++s;
    }
    *v = x;
    return true;
  };
  skip_ws();
  if (*s == '\0') return FP8ATTN_OK;   // empty selector
  for (;;) {
    long lo = 0, hi = 0;
    skip_ws();
    if (!read_int(&lo)) return FP8ATTN_ERR_INVALID;
    hi = lo;
    skip_ws();
    if (*s == '-') {
      ++s;
      skip_ws();
      if (!read_int(&hi)) return FP8ATTN_ERR_INVALID;
      skip_ws();
    }
    if (hi < lo || hi >= max_index) return FP8ATTN_ERR_INVALID;
    for (long i = lo; i <= hi; ++i) mask[static_cast<size_t>(i)] = 1;
    if (*s == ',') { ++s; continue; }
    if (*s == '\0') break;
    return FP8ATTN_ERR_INVALID;
  }
  if (max_index > 0) std::memcpy(mask_out, mask.data(), mask.size());
  return FP8ATTN_OK;
}

int fp8attn_select_mode(const fp8attn_ctx* ctx, const uint8_t* skip_mask, int layer) {
  if (!layer_ok(ctx, layer)) return -1;
  if (skip_mask && skip_mask[layer]) return FP8ATTN_SKIP;
  return ctx->has_static[layer] ? FP8ATTN_STATIC : FP8ATTN_DYNAMIC;
}

int fp8attn_select_mode_at_step(const fp8attn_ctx* ctx, const uint8_t* skip_layers, int layer,
                                const uint8_t* skip_steps, int num_steps, int step) {
  if (!layer_ok(ctx, layer)) return -1;
  if (skip_steps && (step < 0 || step >= num_steps)) return -1;
  if (skip_steps && skip_steps[step]) return FP8ATTN_SKIP;
  return fp8attn_select_mode(ctx, skip_layers, layer);
}

fp8attn_status fp8attn_e4m3_encode(const float* d_in, int64_t n, float scale, void* d_out,
                                   void* stream) {
  if (n < 0 || (n > 0 && (!d_in || !d_out))) return FP8ATTN_ERR_INVALID;
  if (n == 0) return FP8ATTN_OK;
  const cudaError_t e = launch_encode(d_in, n, scale, d_out, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_regroup_heads(const void* d_src, void* d_dst, int64_t tokens,
                                    int num_heads, int groups, int head_bytes, int to_groups,
                                    void* stream) {
  if (tokens < 0 || num_heads < 1 || groups < 1 || head_bytes < 1) return FP8ATTN_ERR_INVALID;
  if (num_heads % groups) return FP8ATTN_ERR_INVALID;
  if (to_groups != 0 && to_groups != 1) return FP8ATTN_ERR_INVALID;
  if (head_bytes % 16) return FP8ATTN_ERR_UNSUPPORTED;
  if (tokens == 0) return FP8ATTN_OK;
  if (!d_src || !d_dst) return FP8ATTN_ERR_INVALID;
  if (!aligned(d_src, 16) || !aligned(d_dst, 16)) return FP8ATTN_ERR_UNSUPPORTED;
  const uintptr_t bytes = static_cast<uintptr_t>(tokens) * num_heads * head_bytes;
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(d_src), d0 = reinterpret_cast<uintptr_t>(d_dst);
  if (s0 < d0 + bytes && d0 < s0 + bytes) return FP8ATTN_ERR_INVALID;   // overlap
  const cudaError_t e = launch_regroup_heads(d_src, d_dst, tokens, num_heads, groups, head_bytes,
                                             to_groups, as_stream(stream));
  if (e != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

const float* fp8attn_static_quant_scale_ptr(fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer) || !ctx->has_static[layer]) return nullptr;
  return ctx->ls[layer].static_qs;
}

const float* fp8attn_static_descale_ptr(fp8attn_ctx* ctx, int layer) {
  if (!layer_ok(ctx, layer) || !ctx->has_static[layer]) return nullptr;
  return ctx->ls[layer].static_ds;
}

fp8attn_status fp8attn_kv_assign_pages(const int32_t* d_seq_lens, const int32_t* d_new_lens,
                                       int rows, int page_size, int32_t* d_block_tables,
                                       int64_t table_stride, int table_width, int32_t* d_owned,
                                       int32_t* d_free_pages, int num_pages, int32_t* d_pool,
                                       int64_t max_tokens, int32_t* d_cu_new, int64_t* d_slots,
                                       int32_t* d_positions, int32_t* d_error, void* stream) {
  if (rows < 0 || num_pages < 1 || table_width < 1 || max_tokens < 0 || page_size < 1)
    return FP8ATTN_ERR_INVALID;
  const int page_log2 = page_log2_of(page_size);
  if (page_log2 < 0 || rows > kMaxPageRows || num_pages >= 1 << 30 || max_tokens > 0x7FFFFFFFLL)
    return FP8ATTN_ERR_UNSUPPORTED;
  if (rows == 0) return max_tokens == 0 ? FP8ATTN_OK : FP8ATTN_ERR_INVALID;
  if (rows > 1 && table_stride < table_width) return FP8ATTN_ERR_INVALID;
  if (!d_seq_lens || !d_new_lens || !d_block_tables || !d_owned || !d_free_pages || !d_pool ||
      !d_cu_new || (max_tokens > 0 && (!d_slots || !d_positions)))
    return FP8ATTN_ERR_INVALID;
  if (!aligned(d_slots, 16) || !aligned(d_positions, 16)) return FP8ATTN_ERR_INVALID;
  AssignPagesLaunch p;
  p.seq = d_seq_lens;
  p.fresh = d_new_lens;
  p.tables = d_block_tables;
  p.table_stride = table_stride;
  p.width = table_width;
  p.owned = d_owned;
  p.free_pages = d_free_pages;
  p.num_pages = num_pages;
  p.pool = d_pool;
  p.rows = rows;
  p.page_log2 = page_log2;
  p.max_tokens = static_cast<int>(max_tokens);
  p.cu = d_cu_new;
  p.slots = d_slots;
  p.positions = d_positions;
  p.err = d_error;
  if (launch_assign_pages(p, as_stream(stream)) != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_kv_write(const void* k, const void* v, int64_t tok_stride,
                                int64_t head_stride, const int64_t* d_slots, int64_t tokens,
                                int num_kv_heads, int head_dim, void* k_cache, void* v_cache,
                                int64_t page_stride, int64_t slot_stride,
                                int64_t cache_head_stride, int num_pages, int page_size,
                                const float* d_quant_scale_qkv, int32_t* d_error, void* stream) {
  if (!d_quant_scale_qkv && tokens > 0) return FP8ATTN_ERR_INVALID;
  return run_kv_write(k, v, tok_stride, head_stride, d_slots, tokens, num_kv_heads, head_dim,
                      k_cache, v_cache, page_stride, slot_stride, cache_head_stride, num_pages,
                      page_size, d_quant_scale_qkv != nullptr, d_quant_scale_qkv, d_error, stream);
}

fp8attn_status fp8attn_kv_write_bf16(const void* k, const void* v, int64_t tok_stride,
                                     int64_t head_stride, const int64_t* d_slots, int64_t tokens,
                                     int num_kv_heads, int head_dim, void* k_cache, void* v_cache,
                                     int64_t page_stride, int64_t slot_stride,
                                     int64_t cache_head_stride, int num_pages, int page_size,
                                     int32_t* d_error, void* stream) {
  return run_kv_write(k, v, tok_stride, head_stride, d_slots, tokens, num_kv_heads, head_dim,
                      k_cache, v_cache, page_stride, slot_stride, cache_head_stride, num_pages,
                      page_size, false, nullptr, d_error, stream);
}

size_t fp8attn_kv_tree_workspace_bytes(int rows, int max_q_len, int max_seqlen, int num_heads,
                                       int num_kv_heads) {
  if (rows < 1 || max_q_len < 1 || max_seqlen < 1 || num_kv_heads < 1 || num_heads < 1 ||
      num_heads % num_kv_heads || rows > kMaxTreeRows)
    return 0;
  return kv_tree_workspace_bytes(rows, max_q_len, max_seqlen, num_heads, num_kv_heads);
}

fp8attn_status fp8attn_kv_tree_fwd(const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                                   const void* k_cache, const void* v_cache,
                                   int64_t page_stride, int64_t slot_stride,
                                   int64_t cache_head_stride, int num_pages, int page_size,
                                   const int32_t* d_block_tables, int64_t table_stride,
                                   int table_width, const int32_t* d_seq_lens,
                                   const int32_t* d_cu_q, int rows, int max_q_len,
                                   int max_seqlen, int64_t total_q, int num_heads,
                                   int num_kv_heads, int head_dim, const float* d_descale_qkv,
                                   const int64_t* d_tree_mask, int mask_words,
                                   float softmax_scale, void* out, void* workspace,
                                   size_t workspace_bytes, int32_t* d_error, void* stream) {
  if (!d_descale_qkv) return FP8ATTN_ERR_INVALID;
  return run_kv_tree(q, q_tok_stride, q_head_stride, k_cache, v_cache, page_stride, slot_stride,
                     cache_head_stride, num_pages, page_size, d_block_tables, table_stride,
                     table_width, d_seq_lens, d_cu_q, rows, max_q_len, max_seqlen, total_q,
                     num_heads, num_kv_heads, head_dim, true, d_descale_qkv, d_tree_mask,
                     mask_words, softmax_scale, out, workspace, workspace_bytes, d_error, stream);
}

fp8attn_status fp8attn_kv_tree_fwd_bf16(const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                                        const void* k_cache, const void* v_cache,
                                        int64_t page_stride, int64_t slot_stride,
                                        int64_t cache_head_stride, int num_pages, int page_size,
                                        const int32_t* d_block_tables, int64_t table_stride,
                                        int table_width, const int32_t* d_seq_lens,
                                        const int32_t* d_cu_q, int rows, int max_q_len,
                                        int max_seqlen, int64_t total_q, int num_heads,
                                        int num_kv_heads, int head_dim,
                                        const int64_t* d_tree_mask, int mask_words,
                                        float softmax_scale, void* out, void* workspace,
                                        size_t workspace_bytes, int32_t* d_error, void* stream) {
  return run_kv_tree(q, q_tok_stride, q_head_stride, k_cache, v_cache, page_stride, slot_stride,
                     cache_head_stride, num_pages, page_size, d_block_tables, table_stride,
                     table_width, d_seq_lens, d_cu_q, rows, max_q_len, max_seqlen, total_q,
                     num_heads, num_kv_heads, head_dim, false, nullptr, d_tree_mask,
                     mask_words, softmax_scale, out, workspace, workspace_bytes, d_error, stream);
}

fp8attn_status fp8attn_selftest_kv_tree_stall(int which, int tile) {
  if (which < 0 || which > 1 || tile < 0) return FP8ATTN_ERR_INVALID;
  stall_next_kv_tree(which == 1, tile);
  return FP8ATTN_OK;
}

fp8attn_status fp8attn_kv_keep_path(void* k_cache, void* v_cache, int64_t page_stride,
                                    int64_t slot_stride, int64_t cache_head_stride, int num_pages,
                                    int page_size, int elem_bytes, int num_kv_heads, int head_dim,
                                    const int32_t* d_block_tables, int64_t table_stride,
                                    int table_width, const int32_t* d_seq_lens,
                                    const int32_t* d_cu_q, int rows, const int32_t* d_paths,
                                    int64_t path_stride, int depth, const int32_t* d_keep_lens,
                                    int32_t* d_error, void* stream) {
  if (rows < 0 || depth < 0 || table_width < 1 || (elem_bytes != 1 && elem_bytes != 2))
    return FP8ATTN_ERR_INVALID;
  KvKeepLaunch p;
  const fp8attn_status st =
      check_cache(k_cache, v_cache, page_stride, slot_stride, cache_head_stride, num_pages,
                  page_size, num_kv_heads, head_dim, elem_bytes == 1, &p.cache);
  if (st != FP8ATTN_OK || rows == 0 || depth == 0) return st;
  if (num_kv_heads >= 1 << 17) return FP8ATTN_ERR_UNSUPPORTED;   // blocks in y
  if (rows > 1 && (table_stride < table_width || path_stride < depth)) return FP8ATTN_ERR_INVALID;
  if (!d_block_tables || !d_seq_lens || !d_cu_q || !d_paths || !d_keep_lens)
    return FP8ATTN_ERR_INVALID;
  p.tables = d_block_tables;
  p.table_stride = table_stride;
  p.width = table_width;
  p.seq = d_seq_lens;
  p.cu = d_cu_q;
  p.rows = rows;
  p.paths = d_paths;
  p.path_stride = path_stride;
  p.depth = depth;
  p.keep = d_keep_lens;
  p.err = d_error;
  if (launch_kv_keep(p, as_stream(stream)) != cudaSuccess) return FP8ATTN_ERR_CUDA;
  g_launches.fetch_add(1);
  return FP8ATTN_OK;
}

uint64_t fp8attn_launch_count(void) { return g_launches.load(); }

}  // extern "C"
