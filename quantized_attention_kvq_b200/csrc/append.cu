// Fused rotate + quantize + pack + append kernel.
//
// One CTA handles the new tokens of one (sequence, kv head) that fall in one
// 64-token-aligned window of the cache; each of its 8 warps takes 8 tokens,
// four lanes per token, lane g of a token owning the 32 channels of
// quantization group g.  Keys: fp64 Walsh-Hadamard butterflies (Dual-QK
// summary Sec. 1; gist.science KQV scheme) or the kv head's key matrix of the
// caller's dual transform pair (Dual-QK Sec. 1, Sec. 3.1), optional bf16 channel 0 (Dual-QK
// Sec. 3.3, App. C.3), per-32-channel asymmetric quantization (Dual-QK
// Sec. 3.3).  Values: the same quantizer, optionally after the same rotation
// and with a clipping ratio on each group's range (Dual-QK App. B.2).
// Both code kinds are staged in shared memory and leave channel-major: key
// words one coalesced row per pruning group, value codes packed into each
// channel's row of the 128-token block.  Only tokens [offset, offset+n_new)
// change (tq-kv incremental cache); value-code words that also hold tokens
// outside that range are read, patched and written back by the one CTA whose
// window contains them.
#include "quantize.cuh"
#include "transform.cuh"

namespace kvq {
namespace {

constexpr int kAppendTile = 64;  // tokens per CTA window, aligned to absolute token positions
constexpr int kAppendWarps = 8;

// 4x4 byte transpose: out[j] byte k = byte j of in[k]
__device__ __forceinline__ void transpose_bytes4(const uint32_t (&in)[4], uint32_t (&out)[4]) {
  const uint32_t t0 = __byte_perm(in[0], in[1], 0x5140), t1 = __byte_perm(in[0], in[1], 0x7362);
  const uint32_t t2 = __byte_perm(in[2], in[3], 0x5140), t3 = __byte_perm(in[2], in[3], 0x7362);
  out[0] = __byte_perm(t0, t2, 0x5410);
  out[1] = __byte_perm(t0, t2, 0x7632);
  out[2] = __byte_perm(t1, t3, 0x5410);
  out[3] = __byte_perm(t1, t3, 0x7632);
}

// Key rows of the window's 64 tokens through the kv head's matrix A of the
// caller's transform pair, as one 64 x 128 x 128 product: channel i of token t
// is the fp64 sum over j = 0..127, in order, of A[i][j] x_tj, rounded to fp32.
// A product of two fp32 numbers is exact in fp64, so a fused multiply-add per
// step rounds once, as a rounded sum of the rounded product does: the result is
// that in-order sum bit for bit.  On entry lane (tt, g) holds channels
// 32g .. 32g+31 of token tt in v; on return the transformed ones.  Every thread
// of the block takes part.  Dynamic shared memory: A^T in fp64 as [j][i]
// (128 KB) and X^T in fp64 as [j][t] (64 KB), token t of row j at column
// (t + 8 (j / 32)) mod 64 so that the four lanes of a token store into
// distinct banks; the fp32 results then take X^T's space as rows [t][i].
constexpr int kPairYStride = kHeadDim + 4;  // floats per token row of the results
constexpr size_t kPairSmemBytes = sizeof(double) * kHeadDim * (kHeadDim + kAppendTile);

__device__ __forceinline__ void transform_rows_block(float (&v)[32], int g, int tt, const float* __restrict__ A,
                                                     double* __restrict__ sA, double* __restrict__ sX) {
  static_assert(kAppendWarps * 32 == 256 && kAppendTile == 64, "thread layout of the product");
#pragma unroll
  for (int r = 0; r < 32; ++r) sX[(32 * g + r) * kAppendTile + ((tt + 8 * g) & (kAppendTile - 1))] = (double)v[r];
  // A^T: thread e converts A[i][4q .. 4q+3], i = e mod 128 (consecutive threads,
  // consecutive i: conflict-free stores)
  const float4* A4 = reinterpret_cast<const float4*>(A);
#pragma unroll 4
  for (int e = threadIdx.x; e < kHeadDim * kHeadDim / 4; e += 256) {
    const int i = e & (kHeadDim - 1), q = e >> 7;
    const float4 m = __ldg(A4 + i * (kHeadDim / 4) + q);
    double* d = sA + 4 * q * kHeadDim + i;
    d[0] = (double)m.x;
    d[kHeadDim] = (double)m.y;
    d[2 * kHeadDim] = (double)m.z;
    d[3 * kHeadDim] = (double)m.w;
  }
  __syncthreads();
  // thread: tokens tb + 16 s (s < 4), channels 8 ib .. 8 ib + 7; a warp reads
  // two A^T addresses (broadcast) and 16 consecutive X^T entries per load
  const int tb = threadIdx.x & 15, ib = threadIdx.x >> 4;
  double acc[4][8];
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int r = 0; r < 8; ++r) acc[s][r] = 0.0;
#pragma unroll 1
  for (int jg = 0; jg < 4; ++jg) {
    int xo[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) xo[s] = (tb + 16 * s + 8 * jg) & (kAppendTile - 1);
#pragma unroll 4
    for (int j = 32 * jg; j < 32 * jg + 32; ++j) {
      const double2* ar = reinterpret_cast<const double2*>(sA + j * kHeadDim + 8 * ib);
      double a[8], x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const double2 p = ar[k];
        a[2 * k] = p.x;
        a[2 * k + 1] = p.y;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) x[s] = sX[j * kAppendTile + xo[s]];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int r = 0; r < 8; ++r) acc[s][r] = __fma_rn(a[r], x[s], acc[s][r]);
    }
  }
  __syncthreads();  // X^T is read: its space takes the results
  float* sY = reinterpret_cast<float*>(sX);
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(sY + (tb + 16 * s) * kPairYStride + 8 * ib + 4 * h) =
          make_float4(__double2float_rn(acc[s][4 * h]), __double2float_rn(acc[s][4 * h + 1]),
                      __double2float_rn(acc[s][4 * h + 2]), __double2float_rn(acc[s][4 * h + 3]));
  __syncthreads();
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const float4 o = *reinterpret_cast<const float4*>(sY + tt * kPairYStride + 32 * g + 4 * m);
    v[4 * m] = o.x;
    v[4 * m + 1] = o.y;
    v[4 * m + 2] = o.z;
    v[4 * m + 3] = o.w;
  }
}

// Rotary embedding of one key row held by four lanes as above, at position
// pos (Dual-QK Sec. 3.4, bucket-relative RoPE): channel i < 64 pairs with
// i + 64, held by lane group g ^ 2; angle pos * inv_freq[i mod 64] in fp64,
// x_i cos - x_{i+64} sin below, x_{i+64} cos + x_i sin above, each product and
// sum rounded once, then rounded to fp32.  All 32 lanes of the warp take part.
__device__ __forceinline__ void rope_row_4lanes(float (&v)[32], int g, int pos, const float* __restrict__ inv_freq) {
  const bool upper = g >= 2;
  const int f0 = 32 * (g & 1);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const double other = (double)__shfl_xor_sync(kFull, v[i], 2);
    double sn, cs;
    sincos(__dmul_rn((double)pos, (double)__ldg(inv_freq + f0 + i)), &sn, &cs);
    const double own = __dmul_rn((double)v[i], cs), cross = __dmul_rn(other, sn);
    v[i] = __double2float_rn(upper ? __dadd_rn(own, cross) : __dsub_rn(own, cross));
  }
}

// bf16 (round to nearest even) copy of this lane's 32 channels into a window row
__device__ __forceinline__ void store_bf16_32(__nv_bfloat16* dst, const float (&v)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// ROT & 3: 0 keys as given, 1 Walsh-Hadamard rotation, 2 the pair's key
// matrix tk[h] (192 KB of dynamic shared memory: one resident block); ROT & 4: keys first rotary-embedded at their token index in the
// view (the offset from their bucket's anchor), frequencies inv_freq
template <int KB, int VB, int ROT, bool CH0, bool ROTV, typename In>
__global__ void __launch_bounds__(kAppendWarps * 32, (ROT & 3) == 2 ? 1 : 3)
    k_quantize_append(AppendArgs a, const float* __restrict__ tk, const float* __restrict__ inv_freq) {
  constexpr int TPW = 32 / VB;            // value tokens per 32-bit word: 8 (INT4) or 16 (INT2)
  constexpr int WPR = kAppendTile / TPW;  // value words per channel in the window: 8 or 4
  // key words [pruning group][token], 16 bits a token (its KB * 4 low bits used)
  __shared__ __align__(16) uint16_t kw[kPruneGroups][kAppendTile + 2];
  // value codes [token][channel], one byte each; rows padded to 144 bytes so
  // that the 16-byte stores of the 8 tokens a quarter-warp holds fall on
  // distinct banks
  __shared__ __align__(16) uint8_t vcode[kAppendTile][kHeadDim + 16];
  // packed value words [word][channel]; rows padded by TPW words so that the
  // TPW-channel x WPR-word block a warp reads falls on distinct banks
  __shared__ __align__(16) uint32_t vword[WPR][kHeadDim + TPW];

  const CacheView& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = blockIdx.z;
  const int w0 = (a.offset / kAppendTile + blockIdx.x) * kAppendTile;  // absolute first token of the window
  const int lo = max(a.offset - w0, 0);                                // window tokens [lo, hi) are new
  const int hi = min(a.offset + a.n_new - w0, kAppendTile);
  const size_t bh = (size_t)b * c.H + h;
  const int tb0 = w0 % kKeyBlock;                                      // window start inside its block: 0 or 64
  const size_t unit_blk = bh * (size_t)(c.cap / kKeyBlock) + w0 / kKeyBlock;  // (unit, block) index
  // four lanes per token, lane group g = lane & 3 holding channels 32g .. 32g+31
  const int g = lane & 3;
  const int tt = warp * 8 + (lane >> 2);  // window token of this lane
  const bool active = tt >= lo && tt < hi;
  // input row of window token tt: (bh * n_new + w0 + tt - offset), never negative when active
  const size_t row = bh * a.n_new + (size_t)(w0 + (active ? tt : lo) - a.offset);
  const In* kin = static_cast<const In*>(a.k_new) + row * kHeadDim + 32 * g;
  const In* vin = static_cast<const In*>(a.v_new) + row * kHeadDim + 32 * g;

  Raw32<In> kraw, vraw;  // value loads issued together with the key loads
  if (active) {
    load_raw(kin, kraw);
    load_raw(vin, vraw);
  } else {
#pragma unroll
    for (int j = 0; j < (int)sizeof(In) * 2; ++j) kraw.w[j] = vraw.w[j] = make_uint4(0, 0, 0, 0);
  }
  float kx[32];
  widen(kraw, kx);

  // ---- key row: rotated, then quantized (keys are not clipped)
  if (ROT & 4) rope_row_4lanes(kx, g, w0 + tt, inv_freq);
  if ((ROT & 3) == 1) rotate_row_4lanes(kx, g, a.inv_sqrt_d);
  if ((ROT & 3) == 2) {
    extern __shared__ __align__(16) double pair_smem[];
    transform_rows_block(kx, g, tt, tk + (size_t)h * kPairElems, pair_smem, pair_smem + kHeadDim * kHeadDim);
  }
  // bf16 window copies (rotated key, then the value below) for tokens with a
  // window slot: every sink token, and of the later tokens only this append's
  // last `recent`, the ones that still own their ring slot when it ends (an
  // earlier token of the same append would race with them for the slot)
  // (positions count from the view's first token: a bucket's anchor with
  // bucket-relative RoPE, whose view's window rows are its sequence's)
  const int wn = c.pos_base + w0 + tt;
  const int wslot = active && (wn < c.sink || wn >= c.pos_base + a.offset + a.n_new - c.recent)
                        ? window_slot(c.sink, c.recent, wn) : -1;
  if (wslot >= 0 &&
      kvq_in_bounds((bh * (size_t)(c.sink + c.recent) + wslot) * kHeadDim + 32 * g, 32, c.win_elems()))
    store_bf16_32(c.kwin + (bh * (size_t)(c.sink + c.recent) + wslot) * kHeadDim + 32 * g, kx);
  uint32_t code[8];
  {
    const bool skip0 = CH0 && g == 0;
    const __half2 sz = quantize_group32<KB>(kx, skip0, 1.0f, code);
#pragma unroll
    for (int p = 0; p < 8; ++p) kw[8 * g + p][tt] = (uint16_t)compress_codes<KB>(code[p]);
    if (active) {
      const size_t ksi = (unit_blk * kGroups + g) * kKeyBlock + tb0 + tt;
      if (kvq_in_bounds(ksi, 1, c.ks_pairs())) c.ks[ksi] = sz;
      if (skip0 && kvq_in_bounds(bh * c.cap + w0 + tt, 1, c.rows())) c.k0[bh * c.cap + w0 + tt] = __float2bfloat16_rn(kx[0]);
    }
  }
  // ---- value row: optionally rotated, the same quantizer with the clipping
  // ratio; codes as bytes, scales token-major
  {
    float vx[32];
    widen(vraw, vx);
    if (ROTV) rotate_row_4lanes(vx, g, a.inv_sqrt_d);
    if (wslot >= 0 &&
        kvq_in_bounds((bh * (size_t)(c.sink + c.recent) + wslot) * kHeadDim + 32 * g, 32, c.win_elems()))
      store_bf16_32(c.vwin + (bh * (size_t)(c.sink + c.recent) + wslot) * kHeadDim + 32 * g, vx);
    const __half2 sz = quantize_group32<VB>(vx, false, c.v_clip, code);
    if (!active) {
#pragma unroll
      for (int p = 0; p < 8; ++p) code[p] = 0;  // tokens outside the append contribute zero bits
    } else if (kvq_in_bounds((bh * c.cap + w0 + tt) * kGroups + g, 1, c.ks_pairs())) {
      c.vs[(bh * c.cap + w0 + tt) * kGroups + g] = sz;
    }
    *reinterpret_cast<uint4*>(&vcode[tt][32 * g]) = make_uint4(code[0], code[1], code[2], code[3]);
    *reinterpret_cast<uint4*>(&vcode[tt][32 * g + 16]) = make_uint4(code[4], code[5], code[6], code[7]);
  }
  __syncthreads();

  // ---- key rows out: one pruning group's run per warp, two tokens a lane
  {
    const int t = 2 * lane;  // window tokens t, t + 1
    const bool a0 = t >= lo && t < hi, a1 = t + 1 >= lo && t + 1 < hi;
    for (int pg = warp; pg < kPruneGroups; pg += kAppendWarps) {
      const size_t idx = (unit_blk * kPruneGroups + pg) * kKeyBlock + tb0 + t;
      const uint32_t w2 = *reinterpret_cast<const uint32_t*>(&kw[pg][t]);  // token t in the low half
      if (!kvq_in_bounds(idx * (KB == 4 ? 2 : 1), KB == 4 ? 4 : 2, c.kc_bytes())) continue;
      if (KB == 4) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(c.kc) + idx;
        if (a0 && a1)
          *reinterpret_cast<uint32_t*>(dst) = w2;
        else if (a0)
          dst[0] = (uint16_t)w2;
        else if (a1)
          dst[1] = (uint16_t)(w2 >> 16);
      } else {
        uint8_t* dst = c.kc + idx;
        const uint32_t b2 = (w2 & 0xFFu) | ((w2 >> 8) & 0xFF00u);
        if (a0 && a1)
          *reinterpret_cast<uint16_t*>(dst) = (uint16_t)b2;
        else if (a0)
          dst[0] = (uint8_t)b2;
        else if (a1)
          dst[1] = (uint8_t)(b2 >> 8);
      }
    }
  }

  // ---- value codes: each thread packs 4 channels x TPW tokens into 4 words
  // (token order, low bits first) with byte transposes
  if (threadIdx.x < 32 * WPR) {
    const int c4 = threadIdx.x & 31, w = threadIdx.x >> 5;  // channels 4 c4 .. 4 c4 + 3, word w
    uint32_t out[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < TPW / 4; ++k) {
      uint32_t in[4], col[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) in[r] = *reinterpret_cast<const uint32_t*>(&vcode[w * TPW + 4 * k + r][4 * c4]);
      transpose_bytes4(in, col);  // col[j]: channel 4 c4 + j, tokens 4k .. 4k + 3
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j] |= compress_codes<VB>(col[j]) << (4 * VB * k);
    }
    *reinterpret_cast<uint4*>(&vword[w][4 * c4]) = make_uint4(out[0], out[1], out[2], out[3]);
  }
  __syncthreads();
  // ...and store them into the channel rows of the 128-token block
  constexpr int TPC = 16 * 8 / VB;  // tokens per 16-byte chunk: 32 or 64
  uint8_t* vblk = c.vc + unit_blk * (size_t)(kHeadDim * (kKeyBlock * VB / 8));
  for (int i = threadIdx.x; i < kHeadDim * WPR; i += blockDim.x) {
    const int ch = i / WPR, w = i % WPR;  // a warp: 32 / WPR channels, all their words
    const int t0 = w * TPW;               // first window token of the word
    const int a0 = max(lo - t0, 0), a1 = min(hi - t0, TPW);  // new tokens of this word: [a0, a1)
    if (a0 >= a1) continue;
    const int tb = tb0 + t0;  // ... inside the block
    const int chunk = (tb / TPC) ^ v_chunk_swizzle(VB, ch);
    uint32_t* dst =
        reinterpret_cast<uint32_t*>(vblk + ch * (kKeyBlock * VB / 8) + chunk * 16 + (tb % TPC) / (8 / VB));
    if (!kvq_in_bounds((size_t)(reinterpret_cast<uint8_t*>(dst) - c.vc), 4, c.vc_bytes())) continue;
    uint32_t word = vword[w][ch];
    if (a0 > 0 || a1 < TPW) {
      const uint32_t keep_lo = a0 * VB >= 32 ? ~0u : ((1u << (a0 * VB)) - 1u);
      const uint32_t keep_hi = a1 * VB >= 32 ? 0u : ~((1u << (a1 * VB)) - 1u);
      word |= *dst & (keep_lo | keep_hi);  // the other tokens' codes stay as they were
    }
    *dst = word;
  }
}

template <int KB, int VB, int ROT, bool CH0, bool ROTV>
cudaError_t launch_typed(const AppendArgs& a, const float* tk, const float* fr, cudaStream_t s) {
  const int first = a.offset / kAppendTile, last = (a.offset + a.n_new - 1) / kAppendTile;
  dim3 grid(last - first + 1, a.c.H, a.c.B);
  dim3 block(kAppendWarps * 32);
  auto kern = a.dtype == KVQ_F32 ? k_quantize_append<KB, VB, ROT, CH0, ROTV, float>
                                 : (a.dtype == KVQ_BF16 ? k_quantize_append<KB, VB, ROT, CH0, ROTV, __nv_bfloat16>
                                                        : k_quantize_append<KB, VB, ROT, CH0, ROTV, __half>);
  const size_t smem = (ROT & 3) == 2 ? kPairSmemBytes : 0;
  if (smem) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, block, smem, s>>>(a, tk, fr);
  return cudaGetLastError();
}

template <int KB, int VB, int ROT, bool ROTV>
cudaError_t launch_ch0(const AppendArgs& a, const float* tk, const float* fr, cudaStream_t s) {
  return a.c.keep_ch0 ? launch_typed<KB, VB, ROT, true, ROTV>(a, tk, fr, s)
                      : launch_typed<KB, VB, ROT, false, ROTV>(a, tk, fr, s);
}

template <int KB, int VB, bool ROTV>
cudaError_t launch_flags(const AppendArgs& a, const float* tk, const float* fr, cudaStream_t s) {
  switch (a.c.rotate + (fr ? 4 : 0)) {
    case 0: return launch_ch0<KB, VB, 0, ROTV>(a, tk, fr, s);
    case 1: return launch_ch0<KB, VB, 1, ROTV>(a, tk, fr, s);
    case 2: return launch_ch0<KB, VB, 2, ROTV>(a, tk, fr, s);
    case 4: return launch_ch0<KB, VB, 4, ROTV>(a, tk, fr, s);
    case 5: return launch_ch0<KB, VB, 5, ROTV>(a, tk, fr, s);
    default: return launch_ch0<KB, VB, 6, ROTV>(a, tk, fr, s);
  }
}

// value rotation is a template flag, so kernels without it stay as small as before
template <int KB, int VB>
cudaError_t launch_bits(const AppendArgs& a, const float* tk, const float* fr, cudaStream_t s) {
  return a.c.rotate_v ? launch_flags<KB, VB, true>(a, tk, fr, s) : launch_flags<KB, VB, false>(a, tk, fr, s);
}

}  // namespace

cudaError_t launch_append_ext(const AppendArgs& a, const float* tk, const float* fr, cudaStream_t s) {
  if (a.c.k_bits == 4 && a.c.v_bits == 4) return launch_bits<4, 4>(a, tk, fr, s);
  if (a.c.k_bits == 4) return launch_bits<4, 2>(a, tk, fr, s);
  if (a.c.v_bits == 4) return launch_bits<2, 4>(a, tk, fr, s);
  return launch_bits<2, 2>(a, tk, fr, s);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) { return launch_append_ext(a, nullptr, nullptr, s); }

KVQ_BOUNDS_COUNTER(bounds_append)

}  // namespace kvq
