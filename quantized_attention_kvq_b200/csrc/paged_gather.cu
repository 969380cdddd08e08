// Dense rows of cached tokens: the mirror of the paged append.
//
// A warp takes 8 tokens of one head's keys (or values), four lanes per token,
// lane g owning 32 channels; a lane reads its codes' bytes, forms
// scale * code + zero with one rounding, takes the row back through the
// transform in fp32 when asked and writes its 32 channels in 16-byte pieces.
#include "paged.cuh"

namespace kvq {
namespace {

constexpr int kGatherWarps = 4;

// Orthonormal Walsh-Hadamard transform of a row held by four lanes, in fp32
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

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16*) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half*) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <int KB, int VB, typename Out>
__global__ void __launch_bounds__(kGatherWarps * 32) k_paged_gather(PagedGatherArgs a) {
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & 3;
  const int tok = (blockIdx.x * kGatherWarps + warp) * 8 + (lane >> 2);
  const int h = blockIdx.y;
  const bool values = a.k == nullptr || blockIdx.z != 0;
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
    const float s = __half2float(reinterpret_cast<const __half*>(blk + lay.ks)[scale_index(t, g)]);
    const float z = __half2float(reinterpret_cast<const __half*>(blk + lay.kz)[k_zero_index(t, g)]);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint8_t* d = blk + k_code_byte(KB, 8 * g + r, t);
      const uint32_t w = KB == 4 ? (uint32_t)d[0] | ((uint32_t)d[2] << 8) : (uint32_t)d[0];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * r + j] = fmaf(s, (float)((w >> (KB * j)) & ((1 << KB) - 1)), z);
    }
    if (c.keep_ch0 && g == 0) x[0] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(blk + lay.k0)[t]);
  } else if (read) {
    const float s = __half2float(reinterpret_cast<const __half*>(blk + lay.vs)[scale_index(t, g)]);
    const float z = __half2float(reinterpret_cast<const __half*>(blk + lay.vz)[scale_index(t, g)]);
    const uint8_t* d = blk + lay.vc + v_token_byte(t);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w = VB == 4 ? (uint32_t)d[(16 * g + 2 * r) * 64] | ((uint32_t)d[(16 * g + 2 * r + 1) * 64] << 8)
                                 : (uint32_t)d[(8 * g + r) * 64];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[4 * r + j] = fmaf(s, (float)((w >> (VB * j)) & ((1 << VB) - 1)), z);
    }
  }
  if (a.rotate_back && (values ? c.rotate_v : c.rotate_k)) rotate_row_4lanes_f32(x, g);
  if (tok >= a.n) return;
  Out* dst = static_cast<Out*>(values ? a.v : a.k) + ((size_t)tok * c.H + h) * kHeadDim + 32 * g;
  uint4* d = reinterpret_cast<uint4*>(dst);
  if constexpr (sizeof(Out) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      d[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                        __float_as_uint(x[4 * i + 3]));
  } else {
    Out* ty = nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = make_uint4(pack2(x[8 * i], x[8 * i + 1], ty), pack2(x[8 * i + 2], x[8 * i + 3], ty),
                        pack2(x[8 * i + 4], x[8 * i + 5], ty), pack2(x[8 * i + 6], x[8 * i + 7], ty));
  }
}

template <int KB, int VB>
cudaError_t launch_typed(const PagedGatherArgs& a, cudaStream_t s) {
  const dim3 grid((a.n + 8 * kGatherWarps - 1) / (8 * kGatherWarps), a.c.H, a.k && a.v ? 2 : 1), block(32 * kGatherWarps);
  if (a.dtype == KVQ_F32)
    k_paged_gather<KB, VB, float><<<grid, block, 0, s>>>(a);
  else if (a.dtype == KVQ_BF16)
    k_paged_gather<KB, VB, __nv_bfloat16><<<grid, block, 0, s>>>(a);
  else
    k_paged_gather<KB, VB, __half><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_gather(const PagedGatherArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 4) return a.c.v_bits == 4 ? launch_typed<4, 4>(a, s) : launch_typed<4, 2>(a, s);
  return a.c.v_bits == 4 ? launch_typed<2, 4>(a, s) : launch_typed<2, 2>(a, s);
}

KVQ_BOUNDS_COUNTER(bounds_paged_gather)

}  // namespace kvq
