// Split decode over the paged cache; instantiated per code width in
// paged_decode_*.cu.
//
// Work split: request b's tiles of 64 tokens for every kv head, in (b, h, tile)
// order, are cut into equal contiguous ranges, one per warp ("rank") of one
// persistent CTA per SM.  A warp works alone: its own ring of shared-memory
// stages filled by bulk async copies, its own online softmax, no barrier with
// other warps; a range leaves one partial per (request, head) it touches, in
// slot unit + rank, and the combine pass joins them.  Consecutive ranks sit on
// different SMs, so a short batch still uses all of them.
//
// Per tile, both products run on the tensor cores straight from the codes:
//   scores  S^T = K Q^T: the key codes are the 16-row operand (16 tokens x 16
//           channels), the query the 8-column one.  A code c under a bit mask is
//           the fp16 subnormal c * 2^-24 (times 4, 16 or 64 at the higher bit
//           fields, taken out again by the query): unpacking costs one AND per
//           two codes and a shift per eight, no conversion.  The query enters as
//           two fp16 pieces, q = hi + lo * 2^-11, in columns of their own.  One
//           accumulator per quantization group, so the per-token scale applies
//           exactly afterwards; the zero-point sums are one more product of the
//           fp16 zeros with the per-group query sums.
//   sums    O^T = V^T P^T: the value codes are the 16-row operand (16 channels x
//           16 tokens), P' = p * scale of the token and group the 8-column one.
//           P' goes from the score layout into the operand layout by an
//           in-register 8x8 transpose; no shared memory is written.
// Softmax: p = 2^(s - M) with M raised only when some p * scale would pass 2^15,
// so P' fits fp16 and one warp vote per tile usually replaces the maxima.  The
// sums over a tile stay in the matrix unit's fp32 accumulators and are then
// added to fp32 registers, so a long sequence does not run up rounding in one
// direction; the zero-point terms are fp32 FMAs.
//
// Precision by output type.  The matrix unit aligns products by their nominal
// exponents, so a subnormal operand costs it as many low bits as the code has
// leading zeros: about 2^-18 of the largest product is lost, nothing beside the
// 2^-8 of a bf16 output.  P' rounded to fp16 errs by 2^-11 of p * scale * code;
// codes counted from their middle (code - 8, code - 2) halve what that
// multiplies, which an fp16 output can tell: there the middle times the
// sum of the rounded P' is subtracted by one more product per group.  For fp32
// outputs the codes become normal fp16 numbers (a mask with an OR of 1024 and
// one subtraction), P' keeps a second fp16 piece, and the value codes are counted
// from their middle before the product, so that nothing cancels.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace kvq {
namespace paged {

using namespace sm100;

constexpr int kSms = 148;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxStages = 6;
constexpr float kMStart = -1.0e30f;    // "no token yet": below any score, finite
constexpr float kLow = 1.0f / 2048.0f;  // weight of a low piece

// query heads per kv head are padded to HC = 4, 8 or 16
// MODE by the output type: how much of P' and of the codes' midpoint is kept
enum { kBf16 = 0, kF16 = 1, kF32 = 2 };

template <int KB, int VB, int HC, int MODE>
struct Shape {
  static constexpr bool PREC = MODE == kF32;
  static constexpr int NT = HC / 4;              // 8-column tiles of the query operand (two pieces per head)
  static constexpr int HT = HC / 4;              // heads per thread
  static constexpr int NP = HC == 4 ? 1 : (HC / 8) * (PREC ? 2 : 1);  // 8-column tiles of P'
  static constexpr bool PAIR = HC == 4 && !PREC;  // P' columns: (head, group of a pair)
  static constexpr int OC = HC == 4 ? 2 : HC / 2;  // fp32 sums per thread and 16-channel tile
  static constexpr int WARPS = 8;
  static constexpr int QF = 8 * NT * 256;         // query fragments: 8 K-steps
  static constexpr int QZ = NT * 128;             // per-group query sums, as a fragment
  static constexpr int QH = HC * 8;               // per head: score factor, channel 0
  static constexpr int WARP_FIXED = QF + QZ + QH;
  static constexpr int FIXED = 260 * 4 + 64 + WARPS * kMaxStages * 8 + WARPS * WARP_FIXED;
  static constexpr int stage(bool ch0) { return BlockLayout(KB, VB, ch0).bytes; }
  static constexpr int stages(bool ch0) {
    const int fit = (kSmemLimit - FIXED - 128) / (WARPS * stage(ch0));
    return fit < kMaxStages ? fit : kMaxStages;
  }
  static constexpr int smem(bool ch0) { return FIXED + 128 + WARPS * stages(ch0) * stage(ch0); }
  static_assert(stages(true) >= 1 && stages(false) >= 1, "ring");
};

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}
// 8x8 transpose of 16-bit elements held two per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 float2_of(uint32_t h2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// two codes under a mask as fp16 pairs: raw subnormals, or (NORMAL) the numbers
// field - MID with field = code times the bit field's factor, exactly: 1024 + field
// is an fp16 whose last place is 1
template <bool NORMAL>
__device__ __forceinline__ uint32_t codes_of(uint32_t w, uint32_t mask, int mid) {
  if (!NORMAL) return w & mask;
  const uint32_t a = (w & mask) | 0x64006400u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), __float2half2_rn(1024.0f + (float)mid));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Bounded wait (about a second); false after a give-up
__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity) {
  if (__builtin_expect(mbar_test_wait(bar, parity), 1)) return true;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 21); ++it)
    if (mbar_try_wait_sleep(bar, parity, 500u)) return true;
  return false;
}

__device__ __forceinline__ int tiles_of(const PagedDecodeArgs& a, int b) {
  const int len = min(max(a.lens[b], 0), a.max_len);
  return (len + kBlockTokens - 1) / kBlockTokens;
}

// What a lane knows of one tile of the warp's range
struct Tile {
  const uint8_t* src;  // its block (nullptr: the page is outside the pool)
  int nval;            // valid tokens, 0..64
  int unit;            // request * H + head, -1 past the range
  uint32_t msk;        // kept channel groups
};

template <int KB, int VB, int HC, int MODE>
__global__ void __launch_bounds__(Shape<KB, VB, HC, MODE>::WARPS * 32, 1) k_paged_decode(PagedDecodeArgs a) {
  using S = Shape<KB, VB, HC, MODE>;
  constexpr bool PREC = S::PREC;
  constexpr int W = S::WARPS, NT = S::NT, HT = S::HT, NP = S::NP, OC = S::OC;
  extern __shared__ __align__(128) uint8_t smem[];
  const PagedView& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  const bool ch0 = c.keep_ch0 != 0;
  const BlockLayout lay(KB, VB, ch0);
  const int ST = S::stages(ch0);

  // ---- tiles per request: chunk prefix sums over the batch
  int* chunk = reinterpret_cast<int*>(smem);  // [257] tiles before each chunk of requests
  int* wtot = chunk + 260;                    // [8]
  const int per_chunk = (a.B + 255) / 256;
  {
    int mine = 0;
    const int b0 = min(tid * per_chunk, a.B), b1 = min(b0 + per_chunk, a.B);
    for (int b = b0; b < b1; ++b) mine += tiles_of(a, b);
    int x = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(kFull, x, m);
      if (lane >= m) x += y;
    }
    if (lane == 31) wtot[warp] = x;
    __syncthreads();
    int before = x - mine;
    for (int w = 0; w < warp; ++w) before += wtot[w];
    chunk[tid] = before;
    if (tid == 255) chunk[256] = before + mine;
    if (blockIdx.x == 0) {  // for the combine
      for (int b = b0; b < b1; ++b) {
        a.starts[b] = before;
        before += tiles_of(a, b);
      }
      if (tid == 255) a.starts[a.B] = chunk[256];
    }
    static_assert(W == 8, "256 threads");
  }
  uint8_t* fix = smem + 260 * 4 + 64;
  const uint32_t bars = smem_addr(fix) + warp * kMaxStages * 8;
  uint8_t* mine = fix + W * kMaxStages * 8 + warp * S::WARP_FIXED;
  uint32_t* qf = reinterpret_cast<uint32_t*>(mine);                  // [8][NT][32] x {b0, b1}
  uint32_t* qz = reinterpret_cast<uint32_t*>(mine + S::QF);          // [NT][32]
  float2* qh = reinterpret_cast<float2*>(mine + S::QF + S::QZ);      // [HC] (factor, channel 0)
  uint8_t* ring = smem + (S::FIXED + 127) / 128 * 128 + (size_t)warp * ST * lay.bytes;
  for (int i = lane; i < S::WARP_FIXED / 4; i += 32) qf[i] = 0;  // columns of absent heads stay zero
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(bars + 8 * s, 1);
    mbar_fence_init();
  }
  __syncthreads();

  const int total = chunk[256] * c.H;
  const int ranks = min(W * kSms, total);
  const int rank = warp * kSms + blockIdx.x;
  if (rank >= ranks) {
    if (lane == 0) a.status[rank] = 0;
    return;
  }
  const int t0 = (int)((long long)rank * total / ranks), n = (int)((long long)(rank + 1) * total / ranks) - t0;

  // ---- one lane looks up one tile, 32 tiles at a time
  auto look_up = [&](int k) {
    Tile d;
    d.src = nullptr;
    d.nval = 0;
    d.unit = -1;
    d.msk = 0;
    const int x = 32 * k + lane;
    if (x >= n) return d;
    const int ti = t0 + x;
    int lo = 0, hi = 256;  // chunk[lo] * H <= ti < chunk[hi] * H
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (chunk[m] * c.H <= ti)
        lo = m;
      else
        hi = m;
    }
    int b = lo * per_chunk, r = ti - chunk[lo] * c.H, tb = tiles_of(a, b);
    while (r >= tb * c.H) {
      r -= tb * c.H;
      tb = tiles_of(a, ++b);
    }
    const int h = r / tb, i = r - h * tb;
    d.unit = b * c.H + h;
    d.nval = min(min(max(a.lens[b], 0), a.max_len) - i * kBlockTokens, kBlockTokens);
    d.msk = a.mask ? a.mask[d.unit] : kFull;
    const int pos = i * kBlockTokens;
    const int page = a.table[(size_t)b * a.max_pages + pos / c.page_tokens];
    if (page >= 0 && page < c.num_pages) {
      const size_t at = c.block_offset(page, h, pos % c.page_tokens);
      if (kvq_in_bounds(at, lay.bytes, c.pool_bytes())) d.src = c.pages + at;
    }
    if (!d.src) d.nval = 0;
    return d;
  };
  Tile cur = look_up(0), nxt = look_up(1);
  int batch = 0;  // index of cur's batch

  constexpr int KROW = kBlockTokens * KB / 2;  // bytes of a key row of 4 channels
  auto issue = [&](int j) {
    const Tile& d = (j >> 5) == batch ? cur : nxt;
    const int from = j & 31;
    const uint8_t* src = reinterpret_cast<const uint8_t*>(__shfl_sync(kFull, reinterpret_cast<uint64_t>(d.src), from));
    const uint32_t msk = __shfl_sync(kFull, d.msk, from);
    const int s = j % ST;
    const uint32_t bar = bars + 8 * s, dst = smem_addr(ring + s * lay.bytes);
    if (src == nullptr) {
      if (lane == 0) mbar_arrive_expect_tx(bar, 0);
      return;
    }
    if (msk == kFull) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, lay.bytes);
        bulk_g2s(dst, src, lay.bytes, bar);
      }
    } else {
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(msk) * KROW + lay.bytes - lay.ks);
      __syncwarp();
      if (((msk >> lane) & 1u) && (lane == 0 || !((msk >> (lane - 1)) & 1u))) {  // a run of kept rows starts here
        const uint32_t rest = ~(msk >> lane);  // msk is not full, so a zero bit follows or the shift brought one
        const int run = __ffs(rest) - 1;
        bulk_g2s(dst + lane * KROW, src + lane * KROW, run * KROW, bar);
      }
      if (lane == 31) bulk_g2s(dst + lay.ks, src + lay.ks, lay.bytes - lay.ks, bar);
    }
  };
  for (int j = 0; j < min(ST, n); ++j) issue(j);

  bool ok = true;
  int unit = -1;
  float M[HT], l[HT], zs[kGroups][HT], O[8][OC], fac[HT], q0[HT];

  constexpr int kTop = PREC ? 6 : 14;
  constexpr float kCode = PREC ? 1.0f : 1.0f / 16777216.0f;  // what a code of 1 is to the matrix unit

  // ---- a segment's query: rotated, masked, split into pieces, as fragments
  auto begin_segment = [&](int u, uint32_t msk) {
    const int b = u / c.H, h = u - b * c.H;
    __syncwarp();
    for (int j = 0; j < a.G; ++j) {
      const size_t at = (size_t)b * a.q_stride + ((size_t)h * a.G + j) * kHeadDim + 4 * lane;
      float x[4];
      if (a.dtype == KVQ_F32)
        load4(static_cast<const float*>(a.q) + at, x);
      else if (a.dtype == KVQ_BF16)
        load4(static_cast<const __nv_bfloat16*>(a.q) + at, x);
      else
        load4(static_cast<const __half*>(a.q) + at, x);
      if (c.rotate_k) {
        float y0 = x[0] + x[1], y1 = x[0] - x[1], y2 = x[2] + x[3], y3 = x[2] - x[3];
        x[0] = y0 + y2;
        x[1] = y1 + y3;
        x[2] = y0 - y2;
        x[3] = y1 - y3;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const float sg = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = fmaf(sg, x[i], __shfl_xor_sync(kFull, x[i], m));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
      }
      const bool sel = (msk >> lane) & 1u;
      float first = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sel ? x[i] : 0.0f;
      if (ch0) {
        first = x[0];
        if (lane == 0) x[0] = 0.0f;
      }
      // a power of two that takes the head's largest channel to [2^14, 2^15)
      // (fp32 outputs, whose codes are not scaled by 2^-24: to [2^6, 2^7))
      const float top = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
      const int ex = top > 0.0f ? min(max(kTop - ilogbf(top), -100), 100) : 0;
      const float up = ldexpf(1.0f, ex);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] *= up;
        sum += x[i];
      }
      // K-steps and columns of this lane's four channels
      const int nt_hi = HC == 16 ? j >> 3 : 0, nt_lo = HC == 4 ? 0 : HC == 8 ? 1 : 2 + (j >> 3);
      const int n_hi = HC == 4 ? 2 * j : j & 7, n_lo = HC == 4 ? 2 * j + 1 : j & 7;
      if (KB == 4) {
        const float y[4] = {x[0], x[2], x[1] * (1.0f / 16.0f), x[3] * (1.0f / 16.0f)};
        float e[4];
        __half hh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hh[i] = __float2half_rn(y[i]);
          e[i] = (y[i] - __half2float(hh[i])) * 2048.0f;
        }
        const int step = lane >> 2, col = lane & 3;
        uint2 v;
        v.x = half2_of(__half2float(hh[0]), __half2float(hh[1]));
        v.y = half2_of(__half2float(hh[2]), __half2float(hh[3]));
        reinterpret_cast<uint2*>(qf)[(step * NT + nt_hi) * 32 + n_hi * 4 + col] = v;
        v.x = half2_of(e[0], e[1]);
        v.y = half2_of(e[2], e[3]);
        reinterpret_cast<uint2*>(qf)[(step * NT + nt_lo) * 32 + n_lo * 4 + col] = v;
      } else {
        const int Q = lane >> 3, col = lane & 3, side = (lane >> 2) & 1;
        __half* qfh = reinterpret_cast<__half*>(qf);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = x[i] * (i == 0 ? 1.0f : i == 1 ? 0.25f : i == 2 ? 0.0625f : 0.015625f);
          const __half hi = __float2half_rn(y);
          const int step = 2 * Q + (i >> 1);
          qfh[(((step * NT + nt_hi) * 32 + n_hi * 4 + col) * 2 + (i & 1)) * 2 + side] = hi;
          qfh[(((step * NT + nt_lo) * 32 + n_lo * 4 + col) * 2 + (i & 1)) * 2 + side] =
              __float2half_rn((y - __half2float(hi)) * 2048.0f);
        }
      }
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) sum += __shfl_xor_sync(kFull, sum, m);
      if ((lane & 7) == 0) {  // group lane / 8: K positions 2 c + b of the zero-point product
        const int Q = lane >> 3;
        const float y = sum * kCode;
        const __half hi = __float2half_rn(y);
        __half* z = reinterpret_cast<__half*>(qz);
        z[(nt_hi * 32 + n_hi * 4 + (Q >> 1)) * 2 + (Q & 1)] = hi;
        z[(nt_lo * 32 + n_lo * 4 + (Q >> 1)) * 2 + (Q & 1)] = __float2half_rn((y - __half2float(hi)) * 2048.0f);
      }
      if (lane == 0) qh[j] = make_float2(a.scale_log2 * ldexpf(1.0f, (PREC ? 0 : 24) - ex), first * up * kCode);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < HT; ++k) {
      const int hd = HC == 4 ? cq : 8 * (k >> 1) + 2 * cq + (k & 1);
      const float2 v = qh[hd];
      fac[k] = v.x;
      q0[k] = v.y;
      M[k] = kMStart;
      l[k] = 0.0f;
#pragma unroll
      for (int r = 0; r < kGroups; ++r) zs[r][k] = 0.0f;
    }
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int r = 0; r < OC; ++r) O[m][r] = 0.0f;
  };

  // ---- a segment's partial: sums over the lanes that share a head, then out
  auto end_segment = [&]() {
#pragma unroll
    for (int k = 0; k < HT; ++k) {
#pragma unroll
      for (int m = 4; m < 32; m <<= 1) {
        l[k] += __shfl_xor_sync(kFull, l[k], m);
#pragma unroll
        for (int r = 0; r < kGroups; ++r) zs[r][k] += __shfl_xor_sync(kFull, zs[r][k], m);
      }
    }
    const float nan = __int_as_float(0x7fc00000);
    constexpr float kOne = 1.0f / kCode;
#pragma unroll
    for (int k = 0; k < HT; ++k) {
      const int hd = HC == 4 ? cq : 8 * (k >> 1) + 2 * cq + (k & 1);
      if (hd >= a.G) continue;
      const size_t row = (size_t)(unit + rank) * a.G + hd;
      if (!kvq_in_bounds(row, 1, a.part_rows)) continue;
      if (g == 0) a.part_ml[row] = ok ? make_float2(M[k], l[k]) : make_float2(nan, nan);
      float* dst = a.part_acc + row * kHeadDim;
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        // rows g and g + 8 of the 16-channel tile m
        const float r0 = HC == 4 ? O[m][0] : O[m][4 * (k >> 1) + (k & 1)];
        const float r1 = HC == 4 ? O[m][1] : O[m][4 * (k >> 1) + 2 + (k & 1)];
        if (VB == 4) {
          float2 v = make_float2(fmaf(r0, kOne, zs[m >> 1][k]), fmaf(r1, kOne / 16.0f, zs[m >> 1][k]));
          *reinterpret_cast<float2*>(dst + 16 * m + 2 * g) = v;
        } else {
          const float s0 = (m & 1) ? kOne / 16.0f : kOne, s1 = (m & 1) ? kOne / 64.0f : kOne / 4.0f;
          float2 v = make_float2(fmaf(r0, s0, zs[m >> 1][k]), fmaf(r1, s1, zs[m >> 1][k]));
          *reinterpret_cast<float2*>(dst + 32 * (m >> 1) + 4 * g + 2 * (m & 1)) = v;
        }
      }
    }
  };

  int s = 0, phase = 0;
  for (int j = 0; j < n; ++j) {
    if ((j >> 5) != batch) {
      ++batch;
      cur = nxt;
      nxt = look_up(batch + 1);
    }
    const int from = j & 31;
    const int u = __shfl_sync(kFull, cur.unit, from);
    const int nval = __shfl_sync(kFull, cur.nval, from);
    if (u != unit) {
      if (unit >= 0) end_segment();
      unit = u;
      begin_segment(u, __shfl_sync(kFull, cur.msk, from));
    }
    if (ok) ok = wait_full(bars + 8 * s, phase);
    ok = __all_sync(kFull, ok);
    if (nval > 0 && ok) {
      const uint8_t* st = ring + s * lay.bytes;
      // ================================================================ scores
      float acc[4][NT][4];
      {
        const uint4 z0 = *reinterpret_cast<const uint4*>(st + lay.kz + (g * 2 + (cq & 1)) * 16);
        const uint4 z1 = *reinterpret_cast<const uint4*>(st + lay.kz + ((8 + g) * 2 + (cq & 1)) * 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t bz = qz[nt * 32 + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][nt][r] = 0.0f;
            const uint4& z = i < 2 ? z0 : z1;
            mma8(acc[i][nt], (i & 1) ? z.z : z.x, (i & 1) ? z.w : z.y, bz);
          }
        }
      }
      uint4 ks[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ks[i] = *reinterpret_cast<const uint4*>(st + lay.ks + 16 * (8 * i + g));
#pragma unroll
      for (int Q = 0; Q < kGroups; ++Q) {
        uint2 bA[NT], bB[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          bA[nt] = reinterpret_cast<const uint2*>(qf)[((2 * Q) * NT + nt) * 32 + lane];
          bB[nt] = reinterpret_cast<const uint2*>(qf)[((2 * Q + 1) * NT + nt) * 32 + lane];
        }
        uint4 w0, w1;
        if (KB == 4) {
          const uint8_t* p = st + (8 * Q + cq) * 128 + 16 * (g ^ (2 * cq));
          w0 = *reinterpret_cast<const uint4*>(p);
          w1 = *reinterpret_cast<const uint4*>(p + 4 * 128);
        } else {
          const uint8_t* p = st + (8 * Q + cq) * 64 + 8 * (g ^ (4 * (cq >> 1)));
          const uint2 x0 = *reinterpret_cast<const uint2*>(p), x1 = *reinterpret_cast<const uint2*>(p + 4 * 64);
          w0 = make_uint4(__byte_perm(x0.x, x1.x, 0x5410), __byte_perm(x0.x, x1.x, 0x7632),
                          __byte_perm(x0.y, x1.y, 0x5410), __byte_perm(x0.y, x1.y, 0x7632));
          w1 = w0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = word(w0, i), y = KB == 4 ? word(w1, i) : x;
          const uint32_t xs = x >> 8, ys = KB == 4 ? y >> 8 : xs;
          constexpr uint32_t m0 = KB == 4 ? 0x000F000Fu : 0x00030003u, m1 = KB == 4 ? 0x00F000F0u : 0x000C000Cu;
          constexpr uint32_t m2 = KB == 4 ? m0 : 0x00300030u, m3 = KB == 4 ? m1 : 0x00C000C0u;
          const uint32_t ka[8] = {codes_of<PREC>(x, m0, 0), codes_of<PREC>(xs, m0, 0), codes_of<PREC>(x, m1, 0),
                                  codes_of<PREC>(xs, m1, 0), codes_of<PREC>(y, m2, 0), codes_of<PREC>(ys, m2, 0),
                                  codes_of<PREC>(y, m3, 0), codes_of<PREC>(ys, m3, 0)};
          const float2 sa = float2_of((Q >> 1) ? ks[i].y : ks[i].x), sb = float2_of((Q >> 1) ? ks[i].w : ks[i].z);
          const float s0 = (Q & 1) ? sa.y : sa.x, s1 = (Q & 1) ? sb.y : sb.x;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma16(d, ka[0], ka[1], ka[2], ka[3], bA[nt].x, bA[nt].y);
            mma16(d, ka[4], ka[5], ka[6], ka[7], bB[nt].x, bB[nt].y);
            acc[i][nt][0] = fmaf(s0, d[0], acc[i][nt][0]);
            acc[i][nt][1] = fmaf(s0, d[1], acc[i][nt][1]);
            acc[i][nt][2] = fmaf(s1, d[2], acc[i][nt][2]);
            acc[i][nt][3] = fmaf(s1, d[3], acc[i][nt][3]);
          }
        }
      }
      // log2-domain scores of this lane's tokens 8g + 2i + e and heads
      float p[4][2][HT];
      {
        uint4 k0 = make_uint4(0, 0, 0, 0);
        if (ch0) k0 = *reinterpret_cast<const uint4*>(st + lay.k0 + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t kk = word(k0, i);
            const float kv = __uint_as_float(e ? kk & 0xFFFF0000u : kk << 16);
            const bool valid = 8 * g + 2 * i + e < nval;
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              float hi, lo;
              if (HC == 4) {
                hi = acc[i][0][2 * e];
                lo = acc[i][0][2 * e + 1];
              } else {
                hi = acc[i][k >> 1][2 * e + (k & 1)];
                lo = acc[i][NT / 2 + (k >> 1)][2 * e + (k & 1)];
              }
              float sc = fmaf(lo, kLow, hi);
              if (ch0) sc = fmaf(q0[k], kv, sc);
              p[i][e][k] = valid ? sc * fac[k] : -INFINITY;
            }
          }
      }
      // ================================================================ softmax
      uint4 vs[4];
      float smax[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vs[i] = *reinterpret_cast<const uint4*>(st + lay.vs + 16 * (8 * i + g));
        if (nval < kBlockTokens) {  // bytes behind the last token may hold anything
          if (8 * g + 2 * i >= nval) vs[i].x = vs[i].y = 0;
          if (8 * g + 2 * i + 1 >= nval) vs[i].z = vs[i].w = 0;
        }
        const __half2 ma = __hmax2(*reinterpret_cast<__half2*>(&vs[i].x), *reinterpret_cast<__half2*>(&vs[i].y));
        const __half2 mb = __hmax2(*reinterpret_cast<__half2*>(&vs[i].z), *reinterpret_cast<__half2*>(&vs[i].w));
        constexpr float kTiny = 1.0f / 16777216.0f;  // the smallest fp16 scale: bounds p where a scale is 0
        smax[i][0] = fmaxf(__half2float(__hmax(__low2half(ma), __high2half(ma))), kTiny);
        smax[i][1] = fmaxf(__half2float(__hmax(__low2half(mb), __high2half(mb))), kTiny);
      }
      {
        // p = 2^(s - M); M rises when some p * scale would pass 2^15
        bool over = false;
        float x[4][2][HT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              x[i][e][k] = ex2(p[i][e][k] - M[k]);
              over |= x[i][e][k] * smax[i][e] > 32768.0f;
            }
        if (__any_sync(kFull, over)) {
#pragma unroll
          for (int k = 0; k < HT; ++k) {
            float t = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) t = fmaxf(t, p[i][e][k] + __log2f(smax[i][e]));
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, m));
            const float m_new = fmaxf(M[k], t - 7.0f);  // the largest P' becomes 2^7: room for 2^8 more
            const float al = ex2(M[k] - m_new);
            M[k] = m_new;
            l[k] *= al;
#pragma unroll
            for (int r = 0; r < kGroups; ++r) zs[r][k] *= al;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              if (HC == 4) {
                O[m][0] *= al;
                O[m][1] *= al;
              } else {
                O[m][4 * (k >> 1) + (k & 1)] *= al;
                O[m][4 * (k >> 1) + 2 + (k & 1)] *= al;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) x[i][e][k] = ex2(p[i][e][k] - m_new);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              p[i][e][k] = x[i][e][k];
              l[k] += x[i][e][k];
            }
      }
      // zero-point terms sum_t p z, per group (codes counted from their middle: z + middle * scale)
      constexpr int kMid = VB == 4 ? 8 : 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 vz = *reinterpret_cast<const uint4*>(st + lay.vz + 16 * (8 * i + g));
        if (nval < kBlockTokens) {
          if (8 * g + 2 * i >= nval) vz.x = vz.y = 0;
          if (8 * g + 2 * i + 1 >= nval) vz.z = vz.w = 0;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float2 z = float2_of(word(vz, 2 * e + r));
            if (MODE != kBf16) {
              const float2 sv = float2_of(word(vs[i], 2 * e + r));
              z.x = fmaf((float)kMid, sv.x, z.x);
              z.y = fmaf((float)kMid, sv.y, z.y);
            }
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              zs[2 * r][k] = fmaf(p[i][e][k], z.x, zs[2 * r][k]);
              zs[2 * r + 1][k] = fmaf(p[i][e][k], z.y, zs[2 * r + 1][k]);
            }
          }
      }
      // ================================================================ value sums
      constexpr int NR = S::PAIR ? 2 : 4;  // rounds: a pair of groups or one group each
#pragma unroll
      for (int rd = 0; rd < NR; ++rd) {
        uint32_t b[4][NP][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (S::PAIR) {
              const float2 sv = float2_of(word(vs[i], 2 * e + rd));
              b[i][0][e] = transpose8(half2_of(p[i][e][0] * sv.x, p[i][e][0] * sv.y));
            } else {
              const float2 s2 = float2_of(word(vs[i], 2 * e + (rd >> 1)));
              const float sv = (rd & 1) ? s2.y : s2.x;
              if (HC == 4) {
                const float v = p[i][e][0] * sv;
                const float hi = __half2float(__float2half_rn(v));
                b[i][0][e] = transpose8(half2_of(hi, (v - hi) * 2048.0f));
              } else {
#pragma unroll
                for (int k = 0; k < HT; k += 2) {
                  const float v0 = p[i][e][k] * sv, v1 = p[i][e][k + 1] * sv;
                  const uint32_t hi = half2_of(v0, v1);
                  b[i][k >> 1][e] = transpose8(hi);
                  if (PREC) {
                    const float2 f = float2_of(hi);
                    b[i][NP / 2 + (k >> 1)][e] = transpose8(half2_of((v0 - f.x) * 2048.0f, (v1 - f.y) * 2048.0f));
                  }
                }
              }
            }
          }
        // minus the codes' middle times the sum of the rounded P' (all rows alike)
        float base[NP][4] = {};
        if (MODE == kF16) {
          constexpr uint32_t c0 = VB == 4 ? 0x80088008u : 0x80028002u, c1 = VB == 4 ? 0x80808080u : 0x80088008u;
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int np = 0; np < NP; ++np) mma16(base[np], c0, c1, c0, c1, b[i][np][0], b[i][np][1]);
        }
        constexpr int MT = S::PAIR ? 4 : 2;  // 16-channel tiles of this round
#pragma unroll
        for (int mm = 0; mm < MT; ++mm) {
          const int m = rd * MT + mm;
          uint4 w;
          if (VB == 4)
            w = *reinterpret_cast<const uint4*>(st + lay.vc + (m * 8 + g) * 64 + cq * 16);
          else
            w = *reinterpret_cast<const uint4*>(st + lay.vc + ((m >> 1) * 8 + g) * 64 + cq * 16);
          float d[NP][4];
#pragma unroll
          for (int np = 0; np < NP; ++np)
#pragma unroll
            for (int r = 0; r < 4; ++r) d[np][r] = (VB == 2 && (m & 1)) ? 16.0f * base[np][r] : base[np][r];
          const uint32_t m0 = VB == 4 ? 0x000F000Fu : (m & 1) ? 0x00300030u : 0x00030003u;
          const uint32_t m1 = VB == 4 ? 0x00F000F0u : (m & 1) ? 0x00C000C0u : 0x000C000Cu;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = word(w, i), xs = x >> 8;
            constexpr int f1 = VB == 4 ? 16 : 4;  // the fields' factors
            const int f = VB == 4 ? 1 : (m & 1) ? 16 : 1;
            const uint32_t a0 = codes_of<PREC>(x, m0, f * kMid), a1 = codes_of<PREC>(x, m1, f * f1 * kMid);
            const uint32_t a2 = codes_of<PREC>(xs, m0, f * kMid), a3 = codes_of<PREC>(xs, m1, f * f1 * kMid);
#pragma unroll
            for (int np = 0; np < NP; ++np) mma16(d[np], a0, a1, a2, a3, b[i][np][0], b[i][np][1]);
          }
          if (S::PAIR) {  // columns of this tile's group of the pair
            const int odd = (m >> 1) & 1;
            O[m][0] += d[0][odd];
            O[m][1] += d[0][2 + odd];
          } else if (HC == 4) {
            O[m][0] += fmaf(d[0][1], kLow, d[0][0]);
            O[m][1] += fmaf(d[0][3], kLow, d[0][2]);
          } else {
#pragma unroll
            for (int t = 0; t < HC / 8; ++t)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                O[m][4 * t + r] += PREC ? fmaf(d[NP / 2 + t][r], kLow, d[t][r]) : d[t][r];
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (j + ST < n && ok) issue(j + ST);
    if (++s == ST) {
      s = 0;
      phase ^= 1;
    }
  }
  end_segment();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) a.status[rank] = ok ? 0 : 1;
  if (!ok) __nanosleep(64000);  // copies still in flight land before the shared memory is given up
}

template <int KB, int VB, int HC, int MODE>
cudaError_t launch_one(const PagedDecodeArgs& a, cudaStream_t s) {
  using S = Shape<KB, VB, HC, MODE>;
  auto kern = k_paged_decode<KB, VB, HC, MODE>;
  const int smem = S::smem(a.c.keep_ch0 != 0);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<kSms, S::WARPS * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <int KB, int VB, int HC>
cudaError_t launch_type(const PagedDecodeArgs& a, cudaStream_t s) {
  if (a.dtype == KVQ_F32) return launch_one<KB, VB, HC, kF32>(a, s);
  return a.dtype == KVQ_F16 ? launch_one<KB, VB, HC, kF16>(a, s) : launch_one<KB, VB, HC, kBf16>(a, s);
}

template <int KB, int VB>
cudaError_t launch_bits(const PagedDecodeArgs& a, cudaStream_t s) {
  if (a.G <= 4) return launch_type<KB, VB, 4>(a, s);
  return a.G <= 8 ? launch_type<KB, VB, 8>(a, s) : launch_type<KB, VB, 16>(a, s);
}

unsigned bounds_44(bool), bounds_42(bool), bounds_24(bool), bounds_22(bool);
cudaError_t launch_44(const PagedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_42(const PagedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_24(const PagedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_22(const PagedDecodeArgs& a, cudaStream_t s);

}  // namespace paged
}  // namespace kvq
