// Quantize new tokens into their slots of the paged cache.
//
// A warp takes 8 tokens of one head's keys (or values), four lanes per token,
// lane g owning the 32 channels of quantization group g: the fp64
// Walsh-Hadamard butterflies and the quantizer of the contiguous append (the
// scale by a reciprocal instead of a division).  Keys and values are separate
// blocks of the grid: twice the parallelism in a decode step's small append, and
// half the registers.
//
// Every byte of a block belongs to one token, so a token's codes go straight from
// the registers to their bytes: no read-modify-write, no staging, no
// agreement between tokens, whatever order the slots come in.
#include "paged.cuh"
#include "quantize.cuh"

namespace kvq {
namespace {

constexpr int kAppendWarps = 4;

template <int KB, int VB, typename In>
__global__ void __launch_bounds__(kAppendWarps * 32) k_paged_append(PagedAppendArgs a) {
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & 3;
  const int tok = (blockIdx.x * kAppendWarps + warp) * 8 + (lane >> 2);
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  const int slot = tok < a.n ? a.slots[tok] : -1;
  const bool active = slot >= 0 && slot < c.slots();
  if (!__any_sync(kFull, active)) return;

  Raw32<In> raw;
  if (active) {
    load_raw(static_cast<const In*>(values ? a.v : a.k) + (size_t)tok * (values ? a.v_stride : a.k_stride) +
                 (size_t)h * kHeadDim + 32 * g, raw);
  } else {
#pragma unroll
    for (int j = 0; j < (int)sizeof(In) * 2; ++j) raw.w[j] = make_uint4(0, 0, 0, 0);
  }
  float x[32];
  widen(raw, x);
  if (values ? c.rotate_v : c.rotate_k) rotate_row_4lanes(x, g, a.inv_sqrt_d);

  const int page = active ? slot / c.page_tokens : 0, off = active ? slot % c.page_tokens : 0;
  const int t = off % kBlockTokens;
  const size_t at = c.block_offset(page, h, off);
  const bool write = active && kvq_in_bounds(at, c.block_bytes, c.pool_bytes());
  uint8_t* blk = c.pages + at;
  const BlockLayout lay(KB, VB, c.keep_ch0 != 0);
  uint32_t code[8];
  if (!values) {
    const bool skip0 = c.keep_ch0 && g == 0;
    const __half2 sz = quantize_group32<KB, true>(x, skip0, 1.0f, code);
    if (!write) return;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w = compress_codes<KB>(code[r]);
      uint8_t* d = blk + k_code_byte(KB, 8 * g + r, t);
      d[0] = (uint8_t)w;
      if (KB == 4) d[2] = (uint8_t)(w >> 8);
    }
    reinterpret_cast<__half*>(blk + lay.ks)[scale_index(t, g)] = __low2half(sz);
    reinterpret_cast<__half*>(blk + lay.kz)[k_zero_index(t, g)] = __high2half(sz);
    if (skip0) reinterpret_cast<__nv_bfloat16*>(blk + lay.k0)[t] = __float2bfloat16_rn(x[0]);
  } else {
    const __half2 sz = quantize_group32<VB, true>(x, false, c.v_clip, code);
    if (!write) return;
    uint8_t* d = blk + lay.vc + v_token_byte(t);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t w = compress_codes<VB>(code[r]);
      if (VB == 4) {
        d[(16 * g + 2 * r) * 64] = (uint8_t)w;
        d[(16 * g + 2 * r + 1) * 64] = (uint8_t)(w >> 8);
      } else {
        d[(8 * g + r) * 64] = (uint8_t)w;
      }
    }
    reinterpret_cast<__half*>(blk + lay.vs)[scale_index(t, g)] = __low2half(sz);
    reinterpret_cast<__half*>(blk + lay.vz)[scale_index(t, g)] = __high2half(sz);
  }
}

template <int KB, int VB>
cudaError_t launch_typed(const PagedAppendArgs& a, cudaStream_t s) {
  const dim3 grid((a.n + 8 * kAppendWarps - 1) / (8 * kAppendWarps), a.c.H, 2), block(32 * kAppendWarps);
  if (a.dtype == KVQ_F32)
    k_paged_append<KB, VB, float><<<grid, block, 0, s>>>(a);
  else if (a.dtype == KVQ_BF16)
    k_paged_append<KB, VB, __nv_bfloat16><<<grid, block, 0, s>>>(a);
  else
    k_paged_append<KB, VB, __half><<<grid, block, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 4) return a.c.v_bits == 4 ? launch_typed<4, 4>(a, s) : launch_typed<4, 2>(a, s);
  return a.c.v_bits == 4 ? launch_typed<2, 4>(a, s) : launch_typed<2, 2>(a, s);
}

KVQ_BOUNDS_COUNTER(bounds_paged_append)

}  // namespace kvq
