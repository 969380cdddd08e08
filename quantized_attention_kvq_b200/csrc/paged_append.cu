// Quantize new tokens into their slots of the paged cache.
//
// A warp takes 8 tokens of one head's keys (or values), four lanes per token,
// lane g owning the 32 channels of quantization group g: fp64 Walsh-Hadamard
// butterflies and the quantizer of the contiguous append: the same bits for the same
// tokens.  Keys and values are separate blocks of the
// grid: twice the parallelism in a decode step's small append, and half the
// registers.
//
// Bound by latencies at 20 warps an SM (64 registers of doubles a lane): 54% of the issue
// slots are used, the fp64 pipe 18%, conversions 22%, memory a quarter.  81 us for 32K
// tokens of 8 heads (INT4 keys, INT2 values; 134 MB in, 30 MB out).  Tried and slower:
// writing words of eight neighbouring tokens instead of bytes (8 us more), persistent
// blocks that fetch their next rows ahead (24 us more).  A rotated row is loaded with its channels
// interleaved over the four lanes, so that five of the seven stages stay in the
// lane; one pass through shared memory (16-byte pieces, swizzled so that both
// sides are free of bank conflicts) then brings lane g its own group, and the
// other two stages stay in the lane too: 32 shared-memory accesses per row and
// lane instead of the 128 shuffles that exchanging doubles takes.
//
// Every byte of a block belongs to one token, so a token's codes go straight from
// the registers to their bytes: no read-modify-write, no staging, no
// agreement between tokens, whatever order the slots come in.
#include "paged.cuh"
#include "quantize.cuh"

namespace kvq {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kAppendBlocks = 5;  // per SM: 96 registers a thread; 6 or 7 spill (121, 131, 152 us with the read-back)

// eight consecutive input elements, widened
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  load4(p, reinterpret_cast<float(&)[4]>(f[0]));
  load4(p + 4, reinterpret_cast<float(&)[4]>(f[4]));
}
template <typename In>
__device__ __forceinline__ void load8(const In* p, float (&f)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  widen2(w.x, (const In*)nullptr, f[0], f[1]);
  widen2(w.y, (const In*)nullptr, f[2], f[3]);
  widen2(w.z, (const In*)nullptr, f[4], f[5]);
  widen2(w.w, (const In*)nullptr, f[6], f[7]);
}

template <int HS, int N>
__device__ __forceinline__ void butterflies(double (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    if ((i & HS) == 0) {
      const double u = x[i], w = x[i + HS];
      x[i] = __dadd_rn(u, w);
      x[i + HS] = __dsub_rn(u, w);
    }
}

// The orthonormal transform of a row, fp64 sums, rounded to fp32: lane g of token
// tt's four leaves with channels 32g .. 32g + 31.  buf: 8 rows of 128 doubles.
// Stages 1, 2, 4, 32, 64 first, then 8 and 16; sums of 16-bit inputs are exact in
// fp64 unless they span more than 2^38, so their order does not show.
template <typename In>
__device__ __forceinline__ void load_rotated(const In* row, int tt, int g, double inv_sqrt_d, double* buf,
                                             float (&v)[32]) {
  double x[32];  // 8k + r: channel 32k + 8g + r
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float f[8];
    load8(row + 32 * k + 8 * g, f);
#pragma unroll
    for (int r = 0; r < 8; ++r) x[8 * k + r] = f[r];
  }
  butterflies<1>(x);
  butterflies<2>(x);
  butterflies<4>(x);
  butterflies<8>(x);   // channels 32 apart
  butterflies<16>(x);  // channels 64 apart
  // piece c of a row (channels 2c, 2c + 1) sits at c with its low three bits changed
  auto place = [&](int c) { return 64 * tt + (c ^ ((c >> 3) & 1) ^ (((c >> 4) & 3) << 1) ^ (3 * (tt & 1))); };
  double2* b2 = reinterpret_cast<double2*>(buf);
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) b2[place(16 * k + 4 * g + j)] = make_double2(x[8 * k + 2 * j], x[8 * k + 2 * j + 1]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const double2 d = b2[place(16 * g + j)];
    x[2 * j] = d.x;
    x[2 * j + 1] = d.y;
  }
  butterflies<8>(x);
  butterflies<16>(x);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __double2float_rn(__dmul_rn(x[i], inv_sqrt_d));
}

template <int KB, int VB, typename In>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendBlocks) k_paged_append(PagedAppendArgs a) {
  __shared__ __align__(16) double rows[kAppendWarps][8 * kHeadDim];
  const PagedView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane & 3;
  const int tok = (blockIdx.x * kAppendWarps + warp) * 8 + (lane >> 2);
  const int h = blockIdx.y;
  const bool values = blockIdx.z != 0;
  let_next_start();
  wait_for_stream();
  const int slot = tok < a.n ? a.slots[tok] : -1;
  const bool active = slot >= 0 && slot < c.slots();
  // the row is loaded beside its slot; lanes behind the last token work on the
  // first one's row, those of skipped tokens on theirs, and write nothing
  const In* row = static_cast<const In*>(values ? a.v : a.k) +
                  (tok < a.n ? (size_t)tok * (values ? a.v_stride : a.k_stride) : (size_t)0) + (size_t)h * kHeadDim;
  float x[32];
  if (values ? c.rotate_v : c.rotate_k) {
    load_rotated(row, lane >> 2, g, a.inv_sqrt_d, rows[warp], x);
  } else {
    Raw32<In> raw;
    load_raw(row + 32 * g, raw);
    widen(raw, x);
  }

  const int page = active ? slot / c.page_tokens : 0, off = active ? slot % c.page_tokens : 0;
  const int t = off % kBlockTokens;
  const size_t at = c.block_offset(page, h, off);
  const bool write = active && kvq_in_bounds(at, c.block_bytes, c.pool_bytes());
  uint8_t* blk = c.pages + at;
  const BlockLayout lay(KB, VB, c.keep_ch0 != 0);
  uint32_t code[8];
  if (!values) {
    const bool skip0 = c.keep_ch0 && g == 0;
    const __half2 sz = quantize_group32_fast<KB>(x, skip0, 1.0f, code);
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
    const __half2 sz = quantize_group32_fast<VB>(x, false, c.v_clip, code);
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
  if (a.dtype == KVQ_F32) return launch_overlapped(k_paged_append<KB, VB, float>, grid, block, 0, s, a);
  if (a.dtype == KVQ_BF16) return launch_overlapped(k_paged_append<KB, VB, __nv_bfloat16>, grid, block, 0, s, a);
  return launch_overlapped(k_paged_append<KB, VB, __half>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 4) return a.c.v_bits == 4 ? launch_typed<4, 4>(a, s) : launch_typed<4, 2>(a, s);
  return a.c.v_bits == 4 ? launch_typed<2, 4>(a, s) : launch_typed<2, 2>(a, s);
}

KVQ_BOUNDS_COUNTER(bounds_paged_append)

}  // namespace kvq
