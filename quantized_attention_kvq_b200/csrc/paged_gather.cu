// Dense rows of cached tokens: the mirror of the paged append.
//
// A warp takes 8 tokens of one head's keys (or values), four lanes per token;
// lane g holds channels 32k + 8g .. 32k + 8g + 7 of every quantization group k,
// so that each store of a warp covers whole 64-byte pieces of its rows (one
// group per lane, which half-writes sectors, measured 43 us where this takes 35:
// 24K tokens of 8 heads, INT4 to bf16 and back through the transform, 132 MB, 3.8
// TB/s).  A lane reads its codes' bytes, forms scale * code + zero with one
// rounding and takes the row back through the transform in fp32 when asked.
// Bound by the loads that follow the slot, 5.7 of the 13 cycles between two instructions
// of a warp, and by the ALU (66%: masks and shifts of codes); 63% of the issue slots are
// used.
#include "paged.cuh"

namespace kvq {
namespace {

constexpr int kGatherWarps = 4;
constexpr int kGatherBlocks = 10;  // per SM: 48 registers a thread (no bound: 56 and 9 blocks, 2 us more for 32K tokens of 8 heads)

// Orthonormal Walsh-Hadamard transform of a row held by four lanes as above, in
// fp32: x[8k + r] is channel 32k + 8g + r, so the stages 1, 2, 4, 32 and 64 stay in
// the lane and 8 and 16 pair lanes g ^ 1 and g ^ 2
__device__ __forceinline__ void rotate_row_4lanes_f32(float (&x)[32], int g) {
#pragma unroll
  for (int hs = 1; hs < 32; hs <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & hs) == 0) {
        const float u = x[i], w = x[i + hs];
        x[i] = u + w;
        x[i + hs] = u - w;
      }
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
    const float sg = (g & m) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = fmaf(sg, x[i], __shfl_xor_sync(kFull, x[i], m));
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
}

// The code at bits [sh, sh + BITS) of a word of at most 16 bits, times 2^sh, as a
// float: under the significand of 2^23 it needs no conversion, only a subtraction
// (and the scale takes 2^-sh)
template <int BITS>
__device__ __forceinline__ float field_of(uint32_t w, int sh) {
  return __uint_as_float((w & (((1u << BITS) - 1u) << sh)) | 0x4B000000u) - 8388608.0f;
}

// four fp16 of one token as floats
__device__ __forceinline__ void halves4(uint2 v, float (&f)[4]) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
  f[0] = a.x;
  f[1] = a.y;
  f[2] = b.x;
  f[3] = b.y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16*) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half*) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int KB, int VB, typename Out>
__global__ void __launch_bounds__(kGatherWarps * 32, kGatherBlocks) k_paged_gather(PagedGatherArgs a) {
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & 3;
  const int tok = (blockIdx.x * kGatherWarps + warp) * 8 + (lane >> 2);
  const int h = blockIdx.y;
  const bool values = a.k == nullptr || blockIdx.z != 0;
  let_next_start();
  wait_for_stream();
  const int slot = tok < a.n ? a.slots[tok] : -1;
  const bool active = slot >= 0 && slot < c.slots();
  const int page = active ? slot / c.page_tokens : 0, off = active ? slot % c.page_tokens : 0;
  const int t = off % kBlockTokens;
  const size_t at = c.block_offset(page, h, off);
  const bool read = active && kvq_in_bounds(at, c.block_bytes, c.pool_bytes());
  const uint8_t* blk = c.pages + at;
  const BlockLayout lay(KB, VB, c.keep_ch0 != 0);
  float x[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = 0.0f;
  if (read && !values) {
    float sc[4], zr[4];
    halves4(*reinterpret_cast<const uint2*>(blk + lay.ks + 2 * scale_index(t, 0)), sc);
    halves4(make_uint2(*reinterpret_cast<const uint32_t*>(blk + lay.kz + 2 * k_zero_index(t, 0)),
                       *reinterpret_cast<const uint32_t*>(blk + lay.kz + 2 * k_zero_index(t, 2))), zr);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* d = blk + k_code_byte(KB, 8 * k + 2 * g + r, t);
        uint32_t w;
        if (KB == 4) {  // the token's two bytes sit in one word
          w = *reinterpret_cast<const uint32_t*>(d - (t & 1)) >> (8 * (t & 1));
          w = __byte_perm(w, 0, 0x4420);
        } else {
          w = d[0];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x[8 * k + 4 * r + j] = fmaf(sc[k] * (1.0f / (1 << (KB * j))), field_of<KB>(w, KB * j), zr[k]);
      }
    if (c.keep_ch0 && g == 0) x[0] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(blk + lay.k0)[t]);
  } else if (read) {
    float sc[4], zr[4];
    halves4(*reinterpret_cast<const uint2*>(blk + lay.vs + 2 * scale_index(t, 0)), sc);
    halves4(*reinterpret_cast<const uint2*>(blk + lay.vz + 2 * scale_index(t, 0)), zr);
    const uint8_t* d = blk + lay.vc + v_token_byte(t);
    constexpr int PER = 8 / VB;  // channels per byte
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int r = 0; r < 8 / PER; ++r) {
        const uint32_t w = d[((32 * k + 8 * g) / PER + r) * 64];
#pragma unroll
        for (int j = 0; j < PER; ++j)
          x[8 * k + PER * r + j] = fmaf(sc[k] * (1.0f / (1 << (VB * j))), field_of<VB>(w, VB * j), zr[k]);
      }
  }
  if (a.rotate_back && (values ? c.rotate_v : c.rotate_k)) rotate_row_4lanes_f32(x, g);
  if (tok >= a.n) return;
  Out* dst = static_cast<Out*>(values ? a.v : a.k) + ((size_t)tok * c.H + h) * kHeadDim + 8 * g;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4* d = reinterpret_cast<uint4*>(dst + 32 * k);
    if constexpr (sizeof(Out) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = make_uint4(__float_as_uint(x[8 * k + 4 * i]), __float_as_uint(x[8 * k + 4 * i + 1]),
                          __float_as_uint(x[8 * k + 4 * i + 2]), __float_as_uint(x[8 * k + 4 * i + 3]));
    } else {
      Out* ty = nullptr;
      d[0] = make_uint4(pack2(x[8 * k], x[8 * k + 1], ty), pack2(x[8 * k + 2], x[8 * k + 3], ty),
                        pack2(x[8 * k + 4], x[8 * k + 5], ty), pack2(x[8 * k + 6], x[8 * k + 7], ty));
    }
  }
}

template <int KB, int VB>
cudaError_t launch_typed(const PagedGatherArgs& a, cudaStream_t s) {
  const dim3 grid((a.n + 8 * kGatherWarps - 1) / (8 * kGatherWarps), a.c.H, a.k && a.v ? 2 : 1), block(32 * kGatherWarps);
  if (a.dtype == KVQ_F32) return launch_overlapped(k_paged_gather<KB, VB, float>, grid, block, 0, s, a);
  if (a.dtype == KVQ_BF16) return launch_overlapped(k_paged_gather<KB, VB, __nv_bfloat16>, grid, block, 0, s, a);
  return launch_overlapped(k_paged_gather<KB, VB, __half>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 4) return a.c.v_bits == 4 ? launch_typed<4, 4>(a, s) : launch_typed<4, 2>(a, s);
  return a.c.v_bits == 4 ? launch_typed<2, 4>(a, s) : launch_typed<2, 2>(a, s);
}

KVQ_BOUNDS_COUNTER(bounds_paged_gather)

}  // namespace kvq
