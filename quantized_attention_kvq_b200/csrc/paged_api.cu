// C ABI of the paged cache: argument checks, workspace carving and launches.
// Every check happens on the host before anything is enqueued; no exception
// leaves this file.
#include <cstdint>

#include "api_util.cuh"
#include "paged.cuh"

namespace kvq {
namespace {

kvq_status check_paged_shape(const kvq_paged_cache* c) {
  if (!c) return KVQ_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_tokens < 1 || c->kv_heads < 1 || c->head_dim < 1) return KVQ_ERR_INVALID_ARG;
  if (c->rotate_k < 0 || c->rotate_k > 2 || (c->keep_ch0 != 0 && c->keep_ch0 != 1)) return KVQ_ERR_INVALID_ARG;
  if ((c->rotate_v != 0 && c->rotate_v != 1) || !(c->v_clip > 0.0f && c->v_clip <= 1.0f)) return KVQ_ERR_INVALID_ARG;
  if (c->rotate_k == 2) return KVQ_ERR_UNSUPPORTED;  // the caller's transform pair: contiguous caches only
  if (c->head_dim != kHeadDim || c->group_size != kGroup || c->prune_granule != kGranule) return KVQ_ERR_UNSUPPORTED;
  if ((c->k_bits != 2 && c->k_bits != 4) || (c->v_bits != 2 && c->v_bits != 4)) return KVQ_ERR_UNSUPPORTED;
  if (c->page_tokens % kBlockTokens != 0 || c->page_tokens > kMaxPageTokens) return KVQ_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * c->page_tokens > INT32_MAX || c->kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * (c->page_tokens / kBlockTokens) * c->kv_heads > INT32_MAX)
    return KVQ_ERR_UNSUPPORTED;  // blocks are numbered in 32 bits (12 TB of pool)
  return KVQ_OK;
}

kvq_status check_paged(const kvq_paged_cache* c) {
  kvq_status st = check_paged_shape(c);
  if (st != KVQ_OK) return st;
  if (!c->pages || (reinterpret_cast<uintptr_t>(c->pages) & 127u) != 0) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

PagedView paged_view(const kvq_paged_cache* c) {
  PagedView v;
  v.num_pages = c->num_pages;
  v.page_tokens = c->page_tokens;
  v.blocks = c->page_tokens / kBlockTokens;
  v.H = c->kv_heads;
  v.k_bits = c->k_bits;
  v.v_bits = c->v_bits;
  v.rotate_k = c->rotate_k;
  v.keep_ch0 = c->keep_ch0;
  v.rotate_v = c->rotate_v;
  v.v_clip = c->v_clip;
  v.pages = static_cast<uint8_t*>(c->pages);
  v.block_bytes = BlockLayout(c->k_bits, c->v_bits, c->keep_ch0 != 0).bytes;
  return v;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Workspace of the paged decode: one partial row (128 sums, running max and
// sum) per (unit + rank, query head of the GQA group), the requests' first
// tiles, and one status word per rank.
struct PagedPlan {
  size_t rows, ml_offset, starts_offset, status_offset, bytes;
};

PagedPlan plan_paged(const kvq_paged_cache* c, int32_t batch, int32_t q_heads) {
  PagedPlan p;
  p.rows = ((size_t)batch * c->kv_heads + kPagedMaxRanks) * (q_heads / c->kv_heads);
  p.ml_offset = round_up(p.rows * kHeadDim * sizeof(float), kAlign);
  p.starts_offset = p.ml_offset + round_up(p.rows * sizeof(float2), kAlign);
  p.status_offset = p.starts_offset + round_up(((size_t)batch + 1) * sizeof(int32_t), kAlign);
  p.bytes = p.status_offset + round_up(kPagedMaxRanks * sizeof(int32_t), kAlign);
  return p;
}

kvq_status check_paged_heads(const kvq_paged_cache* c, int32_t batch, int32_t q_heads) {
  if (batch < 1 || q_heads < 1 || q_heads % c->kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  if (q_heads / c->kv_heads > 16) return KVQ_ERR_UNSUPPORTED;
  if ((int64_t)batch * q_heads > INT32_MAX) return KVQ_ERR_UNSUPPORTED;  // grid of the joining pass
  return KVQ_OK;
}

bool rows_ok(const void* p, int64_t stride, int32_t heads, kvq_dtype dtype) {
  return p && aligned16(p) && stride >= (int64_t)heads * kHeadDim && (stride * (int64_t)dtype_size(dtype)) % 16 == 0;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" {

KVQ_API size_t kvq_paged_bytes(const kvq_paged_cache* c) {
  if (check_paged_shape(c) != KVQ_OK) return 0;
  return paged_view(c).pool_bytes();
}

KVQ_API kvq_status kvq_page_plan(int32_t num_pages, int32_t page_tokens, int32_t batch, const int32_t* ctx_lens,
                                 const int32_t* new_lens, const int32_t* done, int32_t* block_table,
                                 int32_t max_pages, int32_t* free_pages, const int32_t* free_count,
                                 int32_t* free_count_out, int32_t* slots, int32_t* positions, int32_t n_slots,
                                 int32_t* cu_new, int32_t* seq_lens_out, void* stream) {
  NvtxRange range("kvq_page_plan");
  if (num_pages < 1 || page_tokens < 1 || batch < 1 || max_pages < 1 || n_slots < 0) return KVQ_ERR_INVALID_ARG;
  if (!ctx_lens || !new_lens || !block_table || !free_pages || !free_count || !free_count_out || !cu_new ||
      !seq_lens_out || (n_slots > 0 && !slots))
    return KVQ_ERR_INVALID_ARG;
  const void* all[] = {ctx_lens, new_lens, done,      block_table, free_pages,  free_count,
                       free_count_out, slots, positions, cu_new,      seq_lens_out};
  for (const void* p : all)
    if (!aligned4(p)) return KVQ_ERR_INVALID_ARG;
  if (batch > kMaxPlanBatch || n_slots > kMaxRows || page_tokens % kBlockTokens != 0 || page_tokens > kMaxPageTokens ||
      (int64_t)num_pages * page_tokens > INT32_MAX || (int64_t)max_pages * page_tokens > INT32_MAX)
    return KVQ_ERR_UNSUPPORTED;
  PlanArgs a;
  a.page = Divisor(page_tokens);
  a.num_pages = num_pages;
  a.page_tokens = page_tokens;
  a.batch = batch;
  a.max_pages = max_pages;
  a.n_slots = n_slots;
  a.ctx = ctx_lens;
  a.add = new_lens;
  a.done = done;
  a.table = block_table;
  a.free_pages = free_pages;
  a.count = free_count;
  a.count_out = free_count_out;
  a.slots = slots;
  a.positions = positions;
  a.cu = cu_new;
  a.lens = seq_lens_out;
  return cuda_status(launch_page_plan(a, static_cast<cudaStream_t>(stream)));
}

KVQ_API kvq_status kvq_paged_append(const kvq_paged_cache* c, const void* k_new, int64_t k_stride, const void* v_new,
                                    int64_t v_stride, kvq_dtype dtype, int32_t n, const int32_t* slots,
                                    void* stream) {
  NvtxRange range("kvq_paged_append");
  kvq_status st = check_paged(c);
  if (st != KVQ_OK) return st;
  if (!dtype_ok(dtype) || n < 0) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!slots || !aligned4(slots) || !rows_ok(k_new, k_stride, c->kv_heads, dtype) ||
      !rows_ok(v_new, v_stride, c->kv_heads, dtype))
    return KVQ_ERR_INVALID_ARG;
  if (n > kMaxRows) return KVQ_ERR_UNSUPPORTED;
  PagedAppendArgs a;
  a.c = paged_view(c);
  a.k = k_new;
  a.v = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.dtype = dtype;
  a.n = n;
  a.slots = slots;
  a.inv_sqrt_d = inv_sqrt_d();
  return cuda_status(launch_paged_append(a, static_cast<cudaStream_t>(stream)));
}

KVQ_API kvq_status kvq_paged_gather(const kvq_paged_cache* c, const int32_t* slots, int32_t n, kvq_dtype dtype,
                                    int32_t rotate_back, void* k_out, void* v_out, void* stream) {
  NvtxRange range("kvq_paged_gather");
  kvq_status st = check_paged(c);
  if (st != KVQ_OK) return st;
  if (!dtype_ok(dtype) || n < 0 || (rotate_back != 0 && rotate_back != 1)) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (!slots || !aligned4(slots) || (!k_out && !v_out) || !aligned16(k_out) || !aligned16(v_out))
    return KVQ_ERR_INVALID_ARG;
  if (n > kMaxRows) return KVQ_ERR_UNSUPPORTED;
  PagedGatherArgs a;
  a.c = paged_view(c);
  a.slots = slots;
  a.n = n;
  a.dtype = dtype;
  a.rotate_back = rotate_back;
  a.k = k_out;
  a.v = v_out;
  return cuda_status(launch_paged_gather(a, static_cast<cudaStream_t>(stream)));
}

KVQ_API size_t kvq_paged_decode_workspace_bytes(const kvq_paged_cache* c, int32_t batch, int32_t q_heads) {
  if (check_paged_shape(c) != KVQ_OK || check_paged_heads(c, batch, q_heads) != KVQ_OK) return 0;
  return plan_paged(c, batch, q_heads).bytes;
}

KVQ_API kvq_status kvq_paged_decode(const kvq_paged_cache* c, const void* q, int64_t q_stride, kvq_dtype dtype,
                                    int32_t q_heads, int32_t batch, const int32_t* block_table, int32_t max_pages,
                                    const int32_t* seq_lens, int32_t max_len, const uint32_t* mask,
                                    float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  NvtxRange range("kvq_paged_decode");
  kvq_status st = check_paged(c);
  if (st != KVQ_OK) return st;
  if ((st = check_paged_heads(c, batch, q_heads)) != KVQ_OK) return st;
  if (!dtype_ok(dtype) || !rows_ok(q, q_stride, q_heads, dtype) || !block_table || !aligned4(block_table) ||
      !seq_lens || !aligned4(seq_lens) || !aligned4(mask) || !out || !aligned16(out) || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return KVQ_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || max_len < 0 || max_pages < 1) return KVQ_ERR_INVALID_ARG;
  if (max_len > (int64_t)max_pages * c->page_tokens) return KVQ_ERR_CAPACITY;
  const int64_t tiles = ((int64_t)max_len + kBlockTokens - 1) / kBlockTokens;
  if (tiles * batch * c->kv_heads > INT32_MAX) return KVQ_ERR_UNSUPPORTED;  // tiles are counted in 32 bits
  const PagedPlan p = plan_paged(c, batch, q_heads);
  if (workspace_bytes < p.bytes) return KVQ_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  PagedDecodeArgs a;
  a.c = paged_view(c);
  a.q = q;
  a.q_stride = q_stride;
  a.dtype = dtype;
  a.Hq = q_heads;
  a.G = q_heads / c->kv_heads;
  a.B = batch;
  a.max_pages = max_pages;
  a.max_len = max_len;
  a.table = block_table;
  a.lens = seq_lens;
  a.mask = mask;
  a.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);  // log2(e)
  a.out = out;
  a.part_acc = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + p.ml_offset);
  a.starts = reinterpret_cast<int32_t*>(ws + p.starts_offset);
  a.status = reinterpret_cast<int32_t*>(ws + p.status_offset);
  a.part_rows = p.rows;
  a.withheld_tile = take_withheld_tile();
  return cuda_status(launch_paged_decode(a, static_cast<cudaStream_t>(stream)));
}

KVQ_API kvq_status kvq_paged_decode_status(const kvq_paged_cache* c, int32_t batch, int32_t q_heads,
                                           const void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange range("kvq_paged_decode_status");
  kvq_status st = check_paged_shape(c);
  if (st != KVQ_OK) return st;
  if ((st = check_paged_heads(c, batch, q_heads)) != KVQ_OK) return st;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0) return KVQ_ERR_INVALID_ARG;
  const PagedPlan p = plan_paged(c, batch, q_heads);
  if (workspace_bytes < p.bytes) return KVQ_ERR_WORKSPACE;
  int32_t words[kPagedMaxRanks];
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(words, static_cast<const char*>(workspace) + p.status_offset, sizeof(words),
                      cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return KVQ_ERR_CUDA;
  for (int32_t w : words)
    if (w) return KVQ_ERR_TIMEOUT;
  return KVQ_OK;
}

}  // extern "C"
