// Internal helpers of the paged cache: the block layout, the argument blocks of
// the kernels and their launchers (not part of the C ABI).
#pragma once

#include "common.cuh"

namespace kvq {

constexpr int kBlockTokens = 64;    // tokens of one block (one kv head's part of a page, or a piece of it)
constexpr int kScaleBytes = 512;    // one fp16 per token and 32-channel group
constexpr int kMaxPageTokens = 4096;
constexpr int kMaxPlanBatch = 8192;
constexpr int kMaxRows = 1 << 30;  // of one slot list: indexes stay below 2^31

// Byte offsets of a block's parts.  The key codes come first and everything
// else follows in one piece, so that a decode that keeps all channel groups
// copies a block whole and one that does not copies its key rows and the rest.
struct BlockLayout {
  int ks, kz, k0, vc, vs, vz, bytes;
  __host__ __device__ constexpr BlockLayout(int k_bits, int v_bits, bool ch0)
      : ks(kBlockTokens * kHeadDim * k_bits / 8),
        kz(ks + kScaleBytes),
        k0(kz + kScaleBytes),
        vc(k0 + (ch0 ? kBlockTokens * 2 : 0)),
        vs(vc + kBlockTokens * kHeadDim * v_bits / 8),
        vz(vs + kScaleBytes),
        bytes(vz + kScaleBytes) {}
};

// Places inside a block of token t (0..63) = 8u + 2i + e = 16w + 8s + 2i + e.
// The orders are those in which the decode's matrix fragments take the bytes:
// a lane owns the 8 tokens of one u for the scores and the 16 of one w for the
// value sums, and finds them in 16-byte pieces on distinct shared-memory banks.
__host__ __device__ __forceinline__ int k_code_byte(int k_bits, int p, int t) {
  const int u = t >> 3;
  if (k_bits == 4) return p * 128 + 16 * (u ^ (2 * (p & 3))) + 4 * ((t & 7) >> 1) + (t & 1);  // and + 2: channels 4p+2, 4p+3
  return p * 64 + 8 * (u ^ (4 * ((p >> 1) & 1))) + (t & 7);
}
__host__ __device__ __forceinline__ int v_token_byte(int t) {  // of each 64-byte value row
  return 16 * (t >> 4) + 4 * ((t & 7) >> 1) + 2 * ((t >> 3) & 1) + (t & 1);
}
__host__ __device__ __forceinline__ int scale_index(int t, int grp) {  // fp16 units
  return (((((t & 7) >> 1) * 8 + (t >> 3)) * 2 + (t & 1)) << 2) + grp;
}
__host__ __device__ __forceinline__ int k_zero_index(int t, int grp) {  // fp16 units
  const int i = (t & 7) >> 1;
  return (((((i >> 1) * 8 + (t >> 3)) * 2 + (grp >> 1)) * 2 + (i & 1)) * 2 + (t & 1)) * 2 + (grp & 1);
}

struct PagedView {
  int num_pages, page_tokens, blocks;  // blocks = page_tokens / 64 per page and head
  int H, k_bits, v_bits, rotate_k, keep_ch0, rotate_v;
  float v_clip;
  uint8_t* pages;
  int block_bytes;
  __host__ __device__ int slots() const { return num_pages * page_tokens; }
  __host__ __device__ size_t pool_bytes() const { return (size_t)num_pages * H * blocks * block_bytes; }
  // byte offset of the block that holds slot position `off` (0 .. page_tokens - 1) of (page, head h)
  __host__ __device__ size_t block_offset(int page, int h, int off) const {
    return (((size_t)page * H + h) * blocks + off / kBlockTokens) * (size_t)block_bytes;
  }
};

// The paged kernels are launched so that each may take its place on the SMs while
// the kernel before it in the stream drains (programmatic stream serialization):
// wait_for_stream() before the first access to global memory waits until that
// kernel has completed, let_next_start() allows the next one to be placed.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... Args>
cudaError_t launch_overlapped(void (*kern)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// x / d for 0 <= x < 2^31 and 2 <= d < 2^31 by a multiplication: with 2^(l-1) < d <= 2^l,
// m = floor(2^(31+l) / d) + 1 exceeds 2^(31+l) / d by at most 1, which x < 2^31 cannot tell
struct Divisor {
  uint32_t d, m;
  int shift;
  explicit Divisor(int by = 2) : d((uint32_t)by), shift(0) {
    while ((1ull << (shift + 1)) < d) ++shift;
    m = (uint32_t)((1ull << (32 + shift)) / d + 1);
  }
  __device__ __forceinline__ int quotient(int x) const { return (int)(__umulhi((uint32_t)x, m) >> shift); }
};

struct PlanArgs {
  Divisor page;  // by page_tokens
  int num_pages, page_tokens, batch, max_pages, n_slots;
  const int32_t *ctx, *add, *done;
  int32_t *table, *free_pages;
  const int32_t* count;
  int32_t *count_out, *slots, *positions, *cu, *lens;
};
cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s);

struct PagedAppendArgs {
  PagedView c;
  const void *k, *v;
  long long k_stride, v_stride;  // elements between tokens
  int dtype, n;
  const int32_t* slots;
  double inv_sqrt_d;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s);

struct PagedGatherArgs {
  PagedView c;
  const int32_t* slots;
  int n, dtype, rotate_back;
  void *k, *v;
};
cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s);

struct PagedDecodeArgs {
  PagedView c;
  const void* q;
  long long q_stride;
  int dtype, Hq, G, B, max_pages, max_len;
  const int32_t *table, *lens;
  const uint32_t* mask;
  float scale_log2;  // softmax_scale * log2(e): scores live in the exp2 domain
  void* out;
  float* part_acc;   // [units + ranks][G][128] unnormalized sums
  float2* part_ml;   // [units + ranks][G] (running max, running sum)
  int32_t* starts;   // [B + 1] tiles of one kv head before each request
  int32_t* status;   // [kPagedMaxRanks] 1 where a bounded wait of the rank gave up
  int withheld_tile; // test hook: rank 0 never fills this tile's ring slot (-1: none)
  size_t part_rows;
};
// The tiles of a decode are spread over ranks: the warps of one CTA per SM.  More
// warps hide more latency, as long as their registers and rings fit: 8 heads a group
// take 135 us with 12 warps, some 12 more with 14, a number the four schedulers cannot share
// evenly (ragged batch of 64, INT4 / INT2).
constexpr int kPagedSms = 148;
constexpr int paged_decode_warps(int padded_heads, bool f32) {
  return f32 || padded_heads == 16 ? 8 : padded_heads == 8 ? 12 : 16;
}
constexpr int kPagedMaxRanks = 16 * kPagedSms;
inline int paged_decode_ranks(int G, int dtype) {
  return kPagedSms * paged_decode_warps(G <= 4 ? 4 : G <= 8 ? 8 : 16, dtype == KVQ_F32);
}
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t s);

unsigned bounds_paged_append(bool reset);
unsigned bounds_paged_gather(bool reset);
unsigned bounds_paged_decode(bool reset);

}  // namespace kvq
