// Split decode over the paged cache; instantiated per code width in
// paged_decode_*.cu.
//
// Work split: request b's tiles of 64 tokens for every kv head, in (b, h, tile)
// order, are cut into equal contiguous ranges, one per warp ("rank") of one
// persistent CTA per SM.  A warp works alone: its own ring of shared-memory
// stages filled by bulk async copies, its own online softmax, no barrier with
// other warps; a range leaves one partial per (request, head) it touches, in
// slot unit + rank, and a second pass joins them.  Consecutive ranks sit on
// different SMs: a short batch still uses all of them, and requests of many short
// units, which cost more beside their tiles, do not gather on a few (with
// consecutive ranks in one CTA, which then joins its own units, 200 short requests
// measured 44 us where interleaved ranks took 29).
//
// Measured on B200, per call in a stream of calls, both launches (of 6.55 TB/s measured):
// INT4, 8 x 32K tokens, 8 heads of 4 queries 63 us (82%: memory); INT2 with channel 0, 4 x
// 128K 94 us (58%; 61% of the issue slots, ALU 58%, tensor pipe 42%: a third of the
// instructions mask codes out of words, and four warps a scheduler do not cover the waits
// for them and for the products); INT4 / INT2, 64 ragged requests, 8 queries a head 135 us
// (55%; 50% of the issue slots, three warps a scheduler waiting for dependent products); 200
// requests of up to 700 tokens 26 us, of which some 9 are the two launches' fixed part.
// Long fp32 decode (4 x 32K tokens, INT4) 48 us (53%), 16 queries a head (8 x 16K) 44 us (29%):
// 8 warps an SM in both.
//
// Per tile, both products run on the tensor cores straight from the codes:
//   scores  S^T = K Q^T: the key codes are the 16-row operand (16 tokens x 16
//           channels), the query the 8-column one.  A code c under a bit mask is
//           the fp16 subnormal c * 2^-24 (times 4, 16 or 64 at the higher bit
//           fields, taken out again by the query): unpacking costs one AND per
//           two codes and a shift per eight, no conversion.  The query enters as
//           two fp16 pieces, for up to four heads in columns of their own (low pieces
//           times 2^11), for more in products of their own that continue the same
//           sums: half the accumulators.  One
//           accumulator per quantization group, so the per-token scale applies
//           exactly afterwards; the zero-point sums are one more product of the
//           fp16 zeros with the per-group query sums.
//   sums    O^T = V^T P^T: the value codes are the 16-row operand (16 channels x
//           16 tokens), P' = p * scale of the token and group the 8-column one.
//           P' goes from the score layout into the operand layout by an
//           in-register 8x8 transpose; no shared memory is written.
// Softmax: p = 2^(s - M) with M raised only when p or p * scale could pass 2^15
// (bounds kept per warp), so both fit fp16 and one warp vote per tile usually
// replaces the maxima.  p is rounded to fp16 once; P', the zero-point sums, one more
// product with the transposed zeros, and the divisor, a row of ones in it, all start from
// it, so that the rounding of p is that of a weight and not of the output.  The sums over
// a tile stay in the matrix unit's fp32 accumulators and are then added to fp32
// registers, so a long sequence does not run up rounding in one direction.
//
// Precision by output type.  The matrix unit aligns products by their nominal
// exponents, so a subnormal operand costs it as many low bits as the code has
// leading zeros: about 2^-18 of the largest product is lost, nothing beside the
// 2^-8 of a bf16 output.  P' rounded to fp16 errs by 2^-11 of p * scale * code;
// codes counted from their middle (code - 8, code - 2) halve what that
// multiplies, which an fp16 output can tell: there the middle times the
// sum of the rounded P' is subtracted by one more product per group, and the middle
// times the sum of p * scale is added in fp32 (in fp16 that product passes the type's
// range for rotated values whose outputs do not).  For fp32
// outputs the codes become normal fp16 numbers (a mask with an OR of 1024 and
// one subtraction), P' comes from the fp32 p and keeps a second fp16 piece, the
// zero-point sums are fp32 FMAs, and the value codes are counted from their
// middle before the product, so that nothing cancels.
#pragma once

#include <atomic>

#include "paged.cuh"
#include "sm100.cuh"

namespace kvq {
namespace paged {

using namespace sm100;

constexpr int kSms = kPagedSms;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxSlots = 4;            // ring slots of keys, and of values, per warp
constexpr float kMStart = -1.0e30f;     // "no token yet": below any score, finite
constexpr float kLow = 1.0f / 2048.0f;  // weight of a low piece
constexpr float kTop16 = 32768.0f;      // bound of p and of P'

// MODE by the output type: how much of P' and of the codes' middle is kept
enum { kBf16 = 0, kF16 = 1, kF32 = 2 };

// query heads per kv head are padded to HC = 4, 8 or 16
template <int KB, int VB, int HC, int MODE, bool CH0>
struct Shape {
  static constexpr bool PREC = MODE == kF32;
  static constexpr int NT = HC / 4;               // 8-column tiles of the query operand (two pieces per head)
  static constexpr int NA = HC == 4 ? 1 : HC / 8;  // 8-column tiles of scores
  static constexpr float LOW = HC == 4 ? 1.0f / 2048.0f : 1.0f;  // weight of a low piece of the query
  static constexpr int HT = HC / 4;               // heads per thread
  static constexpr int NH = HC == 4 ? 1 : HC / 8;  // 8-column tiles of heads
  static constexpr int NP = NH * (PREC && HC > 4 ? 2 : 1);  // 8-column tiles of P'
  // with a mask, whether only kept key rows are copied: it saves bytes and costs some
  // 100 instructions a tile, so only where bytes are what a decode waits for.
  // INT4 keys and values, 4 heads a group, 32K tokens x 8: 54, 56 and 61 us with 8,
  // 20 and 28 of 32 groups kept against 64 for whole blocks; INT2 at 128K x 4: 94
  // against 88 whatever is kept; INT4 / INT2 with 8 heads a group: 138, 138 and 140
  // with 8, 16 and 24 kept against 132, 134 and 135.
  static constexpr bool PIECES = KB == 4 && HC == 4 && !PREC;
  static constexpr bool PAIR = HC == 4 && !PREC;  // P' columns: (head, group of a pair)
  static constexpr int OC = HC == 4 ? 2 : HC / 2;  // fp32 sums per thread and 16-channel tile
  // whether the divisor is a product of its own with ones: for fp16 outputs no row of the
  // zero-point product is free, and with 8 heads its registers are short (64 ragged
  // requests, INT4 / INT2: 135 us against 138; 4 heads: no difference)
  static constexpr bool ONES = MODE == kF16 || (MODE == kBf16 && HC == 8);
  static constexpr int WARPS = paged_decode_warps(HC, PREC);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int QF = 8 * NT * 256;         // query fragments: 8 K-steps
  static constexpr int QZ = NT * 128;             // per-group query sums, as a fragment
  static constexpr int QH = HC * 8;               // per head: score factor, channel 0
  static constexpr int TILES = 64 * 16;           // what is known of the warp's next tiles
  static constexpr int ROWS = 32;                 // the kept key rows, one byte each
  static constexpr int WARP_FIXED = QF + QZ + QH + TILES + ROWS;
  static constexpr int F_LENS = (THREADS + 4) * 4;  // after the tiles before each chunk of requests: their lengths
  static constexpr int F_WTOT = F_LENS + THREADS * 4;
  static constexpr int F_BARS = F_WTOT + 64;
  static constexpr int F_WARP = F_BARS + WARPS * 2 * kMaxSlots * 8;
  static constexpr int RING = (F_WARP + WARPS * WARP_FIXED + 127) / 128 * 128;
  // a block's two parts: keys (codes, scales, zeros, channel 0) and values
  static constexpr int K_SCALES = BlockLayout(KB, VB, CH0).ks, K_ZEROS = BlockLayout(KB, VB, CH0).kz;
  static constexpr int K_CH0 = BlockLayout(KB, VB, CH0).k0, KPART = BlockLayout(KB, VB, CH0).vc;
  static constexpr int V_SCALES = kBlockTokens * kHeadDim * VB / 8, V_ZEROS = V_SCALES + kScaleBytes;
  static constexpr int VPART = V_ZEROS + kScaleBytes;
  static constexpr int MID = VB == 4 ? 8 : 2;  // the middle of the value codes
  // ring slots per warp: as many as fit, keys first
  static constexpr int slots(bool keys) {
    int k = 1, v = 1;
    const int room = (kSmemLimit - RING) / WARPS;
    while (true) {
      if (k <= v && k < kMaxSlots && (k + 1) * KPART + v * VPART <= room)
        ++k;
      else if (v < k && v < kMaxSlots && k * KPART + (v + 1) * VPART <= room)
        ++v;
      else
        return keys ? k : v;
    }
  }
  static constexpr int SK = slots(true), SV = slots(false);
  static constexpr int WARP_RING = SK * KPART + SV * VPART;
  static constexpr int SMEM = RING + WARPS * WARP_RING;
  static_assert(SMEM <= kSmemLimit, "shared memory");
};

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes global -> shared, asynchronously; the second form arrives on a barrier
// (counted at its initialization) when the thread's copies so far have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// ... from zero
__device__ __forceinline__ void mma16z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma8z(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0), "f"(0.0f));
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
// four 8x8 matrices of 16-bit elements from shared memory, transposed: matrix
// i's rows start at the addresses of lanes 8i .. 8i+7
__device__ __forceinline__ uint4 load_transposed(uint32_t addr) {
  uint4 r;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// one half of a pair in both places
__device__ __forceinline__ uint32_t dup_half(uint32_t a, bool high) {
  const __half2 h = *reinterpret_cast<const __half2*>(&a);
  const __half2 r = high ? __high2half2(h) : __low2half2(h);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
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

// Bounded wait of a whole warp (about a second); false after a give-up
__device__ __forceinline__ bool wait_full(uint32_t bar, uint32_t parity) {
  if (__all_sync(kFull, mbar_test_wait(bar, parity))) return true;
#pragma unroll 1
  for (uint32_t it = 0; it < (1u << 21); ++it)
    if (__all_sync(kFull, mbar_try_wait_sleep(bar, parity, 500u))) return true;
  return false;
}

__device__ __forceinline__ int tiles_of(const PagedDecodeArgs& a, int b) {
  const int len = min(max(a.lens[b], 0), a.max_len);
  return (len + kBlockTokens - 1) / kBlockTokens;
}

// Ranks cut `total` tiles evenly, the first total % ranks taking one tile more
__device__ __forceinline__ int first_tile(int rank, int ranks, int total) {
  const int base = total / ranks;
  return rank * base + min(rank, total - base * ranks);
}
__device__ __forceinline__ int rank_of(int tile, int ranks, int total) {
  const int base = total / ranks, more = total - base * ranks, cut = more * (base + 1);
  return tile < cut ? tile / (base + 1) : more + (tile - cut) / base;
}

// The power of two that value scales up to smax are multiplied with, so that P' = p *
// scale and p both keep their low ends in fp16: 1 for scales of 2^-6 to 2^6.  Smaller ones
// are taken to [1/2, 1): as they are, P' would span as many powers of two fewer above fp16's
// subnormals as they are small, and a long tail of small p be lost.  Larger ones are taken to
// [16, 32), which leaves p 10 of its 15 powers (the bound of p is 2^15 / scale) and small
// scales beside a large one, whose p may be 0, 2^-18 of it before they are subnormal.
__device__ __forceinline__ float scales_up(float smax) {
  if (smax == 0.0f || (smax >= 0.015625f && smax <= 64.0f)) return 1.0f;
  return __int_as_float(((smax < 1.0f ? 253 : 258) - min(__float_as_int(smax) >> 23, 200)) << 23);
}

// One tile of a warp's range, as its lanes leave it in shared memory (16 bytes)
struct Tile {
  int block;     // its block's number in the pool, -1: the page is outside the pool
  int unit;      // request * H + head
  uint32_t msk;  // kept channel groups
  int nval;      // valid tokens, 0..64
};

template <int KB, int VB, int HC, int MODE, bool CH0>
__global__ void __launch_bounds__(Shape<KB, VB, HC, MODE, CH0>::THREADS, 1) k_paged_decode(PagedDecodeArgs a) {
  using S = Shape<KB, VB, HC, MODE, CH0>;
  constexpr bool PREC = S::PREC;
  constexpr int W = S::WARPS, TH = S::THREADS, NT = S::NT, NA = S::NA, HT = S::HT, NH = S::NH, NP = S::NP, OC = S::OC;
  extern __shared__ __align__(128) uint8_t smem[];
  const PagedView& c = a.c;
  // the warp's number through a shuffle: the compiler then knows it to be the same
  // in all lanes, and keeps ring and barrier addresses in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  constexpr int SK = S::SK, SV = S::SV;

  // ---- the requests' tiles: prefix sums over chunks of requests (a chunk is one
  // request up to a batch of TH, whose lengths then stay in shared memory).  The
  // start of the kernel is one chain of memory latencies (lengths, block table,
  // pages), so what does not need the lengths is done while they are on their way.
  int* chunk = reinterpret_cast<int*>(smem);  // [TH + 1] tiles before each chunk
  int* lens_s = reinterpret_cast<int*>(smem + S::F_LENS);
  int* wtot = reinterpret_cast<int*>(smem + S::F_WTOT);
  const int per_chunk = (a.B + TH - 1) / TH;
  const int cb0 = min(tid * per_chunk, a.B), cb1 = min(cb0 + per_chunk, a.B);
  wait_for_stream();
  const int len0 = cb0 < cb1 ? a.lens[cb0] : 0;
  // the block table on its way to L2: each CTA asks for some of its lines
  {
    const long long line = blockIdx.x + (long long)kSms * tid, at = line * 32;  // 32 entries
    if (at < (long long)a.B * a.max_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + at));
  }

  const uint32_t kbars = smem_addr(smem + S::F_BARS) + warp * 2 * kMaxSlots * 8, vbars = kbars + kMaxSlots * 8;
  uint8_t* mine = smem + S::F_WARP + warp * S::WARP_FIXED;
  uint32_t* qf = reinterpret_cast<uint32_t*>(mine);                  // [8][NT][32] x {b0, b1}
  uint32_t* qz = reinterpret_cast<uint32_t*>(mine + S::QF);          // [NT][32]
  float2* qh = reinterpret_cast<float2*>(mine + S::QF + S::QZ);      // [HC] (factor, channel 0)
  Tile* tiles = reinterpret_cast<Tile*>(mine + S::QF + S::QZ + S::QH);  // [64] tiles j at j % 64
  uint8_t* kept = reinterpret_cast<uint8_t*>(tiles + 64);               // [32] kept key rows of the issue's unit
  uint8_t* kring = smem + S::RING + warp * S::WARP_RING;
  uint8_t* vring = kring + SK * S::KPART;
  static_assert(S::WARP_FIXED % 16 == 0 && (S::QF + S::QZ + S::QH) % 16 == 0 && S::F_WARP % 16 == 0, "16-byte stores");
#pragma unroll 4
  for (int i = lane; i < (S::QF + S::QZ + S::QH) / 16; i += 32)  // columns of absent heads stay zero
    reinterpret_cast<uint4*>(mine)[i] = make_uint4(0, 0, 0, 0);
  if (lane == 0) {
    // PIECES: every lane copies key rows and arrives beside the bulk copy of the rest
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(kbars + 8 * s, S::PIECES && a.mask ? 33 : 1);
      mbar_init(vbars + 8 * s, 1);
    }
    mbar_fence_init();
  }
  {
    const int len = min(max(len0, 0), a.max_len);
    lens_s[tid] = len;
    int own = (len + kBlockTokens - 1) / kBlockTokens;
    for (int b = cb0 + 1; b < cb1; ++b) own += tiles_of(a, b);
    int x = own;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(kFull, x, m);
      if (lane >= m) x += y;
    }
    if (lane == 31) wtot[warp] = x;
    __syncthreads();
    int t = lane < W ? wtot[lane] : 0;  // every warp scans the warps' totals for itself
#pragma unroll
    for (int m = 1; m < W; m <<= 1) {
      const int y = __shfl_up_sync(kFull, t, m);
      if (lane >= m) t += y;
    }
    const int prev = __shfl_sync(kFull, t, (warp + 31) & 31);
    int before = x - own + (warp > 0 ? prev : 0);
    chunk[tid] = before;
    if (tid == TH - 1) chunk[TH] = before + own;
    if (blockIdx.x == 0) {  // for the combine
      for (int b = cb0; b < cb1; ++b) {
        a.starts[b] = before;
        before += tiles_of(a, b);
      }
      if (tid == TH - 1) a.starts[a.B] = chunk[TH];
    }
    if (warp == 0 && lane == 0)  // status words of ranks other shapes have
      for (int r = W * kSms + blockIdx.x; r < kPagedMaxRanks; r += kSms) a.status[r] = 0;
  }
  __syncthreads();

  const int total = chunk[TH] * c.H;
  const int ranks = min(W * kSms, total);
  const int rank = warp * kSms + blockIdx.x;
  if (rank >= ranks) {
    if (lane == 0) a.status[rank] = 0;
    return;
  }
  const int t0 = first_tile(rank, ranks, total), n = first_tile(rank + 1, ranks, total) - t0;

  // ---- one lane looks up one tile, 32 tiles at a time
  auto look_up = [&](int k) {
    const int x = 32 * k + lane;
    if (x < n) {
      const int ti = t0 + x;
      int lo = 0, hi = TH;  // chunk[lo] * H <= ti < chunk[hi] * H
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (chunk[m] * c.H <= ti)
          lo = m;
        else
          hi = m;
      }
      int b = lo * per_chunk, r = ti - chunk[lo] * c.H, tb, len;
      if (per_chunk == 1) {
        tb = chunk[lo + 1] - chunk[lo];
        len = lens_s[lo];
      } else {
        tb = tiles_of(a, b);
        while (r >= tb * c.H) {
          r -= tb * c.H;
          tb = tiles_of(a, ++b);
        }
        len = min(max(a.lens[b], 0), a.max_len);
      }
      const int h = r / tb, pos = (r - h * tb) * kBlockTokens;
      Tile d;
      d.unit = b * c.H + h;
      d.nval = min(len - pos, kBlockTokens);
      d.msk = a.mask ? a.mask[d.unit] : kFull;
      const int pg = pos / c.page_tokens;
      const int page = a.table[(size_t)b * a.max_pages + pg];
      d.block = -1;
      if (page >= 0 && page < c.num_pages) d.block = (page * c.H + h) * c.blocks + (pos - pg * c.page_tokens) / kBlockTokens;
      if (d.block >= 0 && !kvq_in_bounds((size_t)d.block * c.block_bytes, c.block_bytes, c.pool_bytes())) d.block = -1;
      if (d.block < 0) d.nval = 0;
      tiles[x & 63] = d;
    }
    __syncwarp();
  };
  look_up(0);

  // ---- ring copies.  A block's key part is one bulk copy.  PIECES with a mask: its
  // kept rows are spread over the lanes in 16-byte pieces (a bulk copy per run of
  // rows costs some 15 instructions each, issued one lane at a time); lane's
  // q-th piece is piece 32 q + lane of the kept rows, and where the pieces are
  // changes with the unit only.
  constexpr int KROW = kBlockTokens * KB / 2;  // bytes of a key row of 4 channels
  constexpr int PPR = KROW / 16, NPC = PPR;  // pieces per row, and per lane
  uint32_t run_msk = kFull;
  int n_pieces = 32 * PPR;
  uint32_t rows_of[(NPC + 3) / 4];  // the row of each of the lane's pieces, a byte each (registers are short)
#pragma unroll
  for (int q = 0; q < NPC; ++q)
    rows_of[q >> 2] = (q & 3 ? rows_of[q >> 2] : 0) | (uint32_t)((32 * q + lane) / PPR) << (8 * (q & 3));
  auto issue_keys = [&](int j, int s) {
    const Tile d = tiles[j & 63];
    const uint32_t bar = kbars + 8 * s, dst = smem_addr(kring + s * S::KPART);
    const uint8_t* src = c.pages + (size_t)d.block * c.block_bytes;
    if (!S::PIECES || !a.mask) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, d.block >= 0 ? S::KPART : 0);
        if (d.block >= 0) bulk_g2s(dst, src, S::KPART, bar);
      }
      return;
    }
    if (d.msk != run_msk) {
      run_msk = d.msk;
      n_pieces = __popc(run_msk) * PPR;
      if ((run_msk >> lane) & 1u) kept[__popc(run_msk & ((1u << lane) - 1u))] = (uint8_t)lane;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < NPC; ++q)
        rows_of[q >> 2] = (q & 3 ? rows_of[q >> 2] : 0) | (uint32_t)kept[min((32 * q + lane) / PPR, 31)] << (8 * (q & 3));
      __syncwarp();
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, d.block >= 0 ? S::KPART - S::K_SCALES : 0);
      if (d.block >= 0) bulk_g2s(dst + S::K_SCALES, src + S::K_SCALES, S::KPART - S::K_SCALES, bar);
    }
    if (d.block >= 0) {
#pragma unroll
      for (int q = 0; q < NPC; ++q)
        if (32 * q + lane < n_pieces) {
          const uint32_t at = ((rows_of[q >> 2] >> (8 * (q & 3))) & 31u) * KROW + (lane & (PPR - 1)) * 16;
          copy16(dst + at, src + at);
        }
    }
    copies_arrive(bar);
  };
  auto issue_values = [&](int j, int s) {
    if (lane == 0) {
      if (j == a.withheld_tile && rank == 0) return;
      const int block = tiles[j & 63].block;
      mbar_arrive_expect_tx(vbars + 8 * s, block >= 0 ? S::VPART : 0);
      if (block >= 0)
        bulk_g2s(smem_addr(vring + s * S::VPART), c.pages + (size_t)block * c.block_bytes + S::KPART, S::VPART, vbars + 8 * s);
    }
  };
  // a segment's query rows as they come.  The first segment's are asked for before
  // the ring's first copies: behind them they would wait for some 20 MB (8000
  // cycles were measured), and no score can start without them.
  constexpr int PASSES = HC / 4, QW = MODE == kF32 ? 4 : 2;  // 16-byte words per lane and pass
  struct QueryRaw {
    uint4 w[QW];
  } raw0[PASSES];
  auto load_query = [&](int u, QueryRaw (&raw)[PASSES]) {
    const int b = u / c.H, h = u - b * c.H;
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      const int j = 4 * ps + (lane >> 3);
      const size_t at = (size_t)b * a.q_stride + ((size_t)h * a.G + (j < a.G ? j : 0)) * kHeadDim + 16 * (lane & 7);
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.q) + at * (MODE == kF32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < QW; ++i) raw[ps].w[i] = p[i];
    }
  };
  load_query(tiles[0].unit, raw0);
#pragma unroll 1
  for (int j = 0; j < min(max(SK, SV), n); ++j) {
    if (j < SK) issue_keys(j, j);
    if (j < SV) issue_values(j, j);
  }

  int unit = tiles[0].unit;
  float M[HT], l[HT], O[8][OC];
  // zero-point sums: per group and head of the thread's own tokens (fp32), or
  // as the product with the zeros leaves them (rows: groups)
  float zs[kGroups][HT], zp[NH][4];
  // largest value scale met, power of two that the scales are multiplied with (P' and O
  // carry it), bound of p that keeps P' in fp16
  float smax = 0.0f, up = 1.0f, plim = kTop16;

  constexpr int kTop = PREC ? 6 : 14;
  constexpr float kUp = 1.0f / S::LOW;
  constexpr float kCode = PREC ? 1.0f : 1.0f / 16777216.0f;  // what a code of 1 is to the matrix unit

  // ---- a segment's query: rotated, masked, split into pieces, as fragments.
  // Four heads at a time, eight lanes per head, a lane holding 16 channels: few
  // shuffles and short chains, since no score can start before it is done.
  auto prepare_query = [&](int u, uint32_t msk, QueryRaw (&raw)[PASSES]) {
    __syncwarp();
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
      if (4 * ps >= a.G) break;
      const int j = 4 * ps + (lane >> 3), part = lane & 7;  // channels 16 part .. 16 part + 15
      const bool live = j < a.G;
      float x[16];
#pragma unroll
      for (int i = 0; i < QW; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t u32 = word(raw[ps].w[i], r);
          if (MODE == kF32) {
            x[4 * i + r] = __uint_as_float(u32);
          } else {
            const float2 f = MODE == kBf16 ? make_float2(__uint_as_float(u32 << 16), __uint_as_float(u32 & 0xFFFF0000u)) : float2_of(u32);
            x[(8 * i + 2 * r) & 15] = f.x;
            x[(8 * i + 2 * r + 1) & 15] = f.y;
          }
        }
      if (c.rotate_k) {
#pragma unroll
        for (int hs = 1; hs < 16; hs <<= 1)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((i & hs) == 0) {
              const float y0 = x[i] + x[i + hs], y1 = x[i] - x[i + hs];
              x[i] = y0;
              x[i + hs] = y1;
            }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) {
          const float sg = (lane & m) ? -1.0f : 1.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = fmaf(sg, x[i], __shfl_xor_sync(kFull, x[i], m));
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
      }
      float first = 0.0f, top = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = ((msk >> (4 * part + (i >> 2))) & 1u) ? x[i] : 0.0f;
      if (CH0) {
        first = x[0];  // of part 0
        if (part == 0) x[0] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
      // a power of two that takes the head's largest channel to [2^14, 2^15)
      // (fp32 outputs, whose codes are not scaled by 2^-24: to [2^6, 2^7))
#pragma unroll
      for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
      const int ex = min(max(kTop + 127 - (__float_as_int(top) >> 23), -100), 100);
      const float up = __int_as_float((127 + ex) << 23);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] *= up;
        sum += x[i];
      }
      sum += __shfl_xor_sync(kFull, sum, 1);  // two lanes hold a quantization group
      // K-steps and columns of this lane's four channel groups p = 4 part + i
      const int nt_hi = HC == 16 ? j >> 3 : 0, nt_lo = HC == 4 ? 0 : HC == 8 ? 1 : 2 + (j >> 3);
      const int n_hi = HC == 4 ? 2 * j : j & 7, n_lo = HC == 4 ? 2 * j + 1 : j & 7;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4], e[4];
        if (KB == 4) {  // (channels 0, 2), (1, 3) / 16, minus what a whole byte brings of the upper field
          y[0] = x[4 * i];
          y[1] = x[4 * i + 2];
          y[2] = x[4 * i + 1] * (1.0f / 16.0f) - (PREC ? 0.0f : y[0]);
          y[3] = x[4 * i + 3] * (1.0f / 16.0f) - (PREC ? 0.0f : y[1]);
        } else {
          y[0] = x[4 * i];
          y[1] = x[4 * i + 1] * 0.25f;
          y[2] = x[4 * i + 2] * 0.0625f;
          y[3] = x[4 * i + 3] * 0.015625f;
        }
        const uint32_t h01 = half2_of(y[0], y[1]), h23 = half2_of(y[2], y[3]);
        const float2 f01 = float2_of(h01), f23 = float2_of(h23);
        e[0] = (y[0] - f01.x) * kUp;
        e[1] = (y[1] - f01.y) * kUp;
        e[2] = (y[2] - f23.x) * kUp;
        e[3] = (y[3] - f23.y) * kUp;
        const uint32_t l01 = half2_of(e[0], e[1]), l23 = half2_of(e[2], e[3]);
        if (KB == 4) {  // step part, column i
          if (live) {
            reinterpret_cast<uint2*>(qf)[(part * NT + nt_hi) * 32 + n_hi * 4 + i] = make_uint2(h01, h23);
            reinterpret_cast<uint2*>(qf)[(part * NT + nt_lo) * 32 + n_lo * 4 + i] = make_uint2(l01, l23);
          }
        } else {
          // steps 2 Q (channels 0, 1) and 2 Q + 1 (channels 2, 3), column i; a word's
          // low half is of the even lane's group, its high half of the odd lane's:
          // the even lane writes the high pieces of both, the odd one the low pieces
          const bool odd = part & 1;
          const uint32_t own01 = odd ? l01 : h01, own23 = odd ? l23 : h23;
          const uint32_t got01 = __shfl_xor_sync(kFull, odd ? h01 : l01, 1), got23 = __shfl_xor_sync(kFull, odd ? h23 : l23, 1);
          const uint32_t e01 = odd ? got01 : own01, o01 = odd ? own01 : got01, e23 = odd ? got23 : own23, o23 = odd ? own23 : got23;
          if (live) {
            uint2* q2 = reinterpret_cast<uint2*>(qf) + ((part & ~1) * NT + (odd ? nt_lo : nt_hi)) * 32 + (odd ? n_lo : n_hi) * 4 + i;
            q2[0] = make_uint2(__byte_perm(e01, o01, 0x5410), __byte_perm(e01, o01, 0x7632));
            q2[NT * 32] = make_uint2(__byte_perm(e23, o23, 0x5410), __byte_perm(e23, o23, 0x7632));
          }
        }
      }
      if (live) {
        if ((part & 1) == 0) {  // group part / 2: K positions 2 c + b of the zero-point product
          const int Q = part >> 1;
          const float y = sum * kCode;
          const __half hi = __float2half_rn(y);
          __half* z = reinterpret_cast<__half*>(qz);
          z[(nt_hi * 32 + n_hi * 4 + (Q >> 1)) * 2 + (Q & 1)] = hi;
          z[(nt_lo * 32 + n_lo * 4 + (Q >> 1)) * 2 + (Q & 1)] = __float2half_rn((y - __half2float(hi)) * kUp);
        }
        if (part == 0) {
          const float f = a.scale_log2 * __int_as_float((127 + (PREC ? 0 : 24) - ex) << 23);
          // a scale of 0 still tells masked tokens (-inf) from the others
          qh[j] = make_float2(f == 0.0f ? 1.0e-37f : f, first * up * kCode);
        }
      }
    }
    __syncwarp();
    smax = 0.0f;
    up = 1.0f;
    plim = kTop16;
#pragma unroll
    for (int k = 0; k < HT; ++k) {
      M[k] = kMStart;
      l[k] = 0.0f;
#pragma unroll
      for (int r = 0; r < kGroups; ++r) zs[r][k] = 0.0f;
    }
#pragma unroll
    for (int t = 0; t < NH; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) zp[t][r] = 0.0f;
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
      for (int r = 0; r < OC; ++r) O[m][r] = 0.0f;
  };

  // the heads of this thread's columns (and, for absent heads, nothing that is used)
  auto head_of = [&](int k) { return HC == 4 ? cq : 8 * (k >> 1) + 2 * cq + (k & 1); };

  // ---- a segment's partial: sums over the lanes that share a head, then out
  auto end_segment = [&]() {
#pragma unroll
    for (int k = 0; k < HT; ++k) {
      if (PREC) {
#pragma unroll
        for (int m = 4; m < 32; m <<= 1) {
          l[k] += __shfl_xor_sync(kFull, l[k], m);
#pragma unroll
          for (int r = 0; r < kGroups; ++r) zs[r][k] += __shfl_xor_sync(kFull, zs[r][k], m);
        }
      }
      if (!PREC && !S::ONES) l[k] = __shfl_sync(kFull, zp[k >> 1][k & 1], 16 + cq);
      if (!PREC) {  // group r: row r (even tokens) and row 12 + r (odd ones) of the zeros' product
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          const float lo = zp[k >> 1][k & 1], hi = zp[k >> 1][2 + (k & 1)];
          zs[r][k] = __shfl_sync(kFull, lo, 4 * r + cq) + __shfl_sync(kFull, hi, 16 + 4 * r + cq);
          if (MODE == kF16)  // and the codes' middle times the scales' sums
            zs[r][k] = fmaf(S::MID, __shfl_sync(kFull, hi, 4 * r + cq) + __shfl_sync(kFull, lo, 16 + 4 * r + cq), zs[r][k]);
        }
      }
    }
    const float one = 1.0f / (kCode * up);
#pragma unroll
    for (int k = 0; k < HT; ++k) {
      const int hd = head_of(k);
      if (hd >= a.G) continue;
      const size_t row = (size_t)(unit + rank) * a.G + hd;
      if (!kvq_in_bounds(row, 1, a.part_rows)) continue;
      if (g == 0) a.part_ml[row] = make_float2(M[k], l[k]);
      float* dst = a.part_acc + row * kHeadDim;
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        // rows g and g + 8 of the 16-channel tile m
        const float r0 = HC == 4 ? O[m][0] : O[m][4 * (k >> 1) + (k & 1)];
        const float r1 = HC == 4 ? O[m][1] : O[m][4 * (k >> 1) + 2 + (k & 1)];
        if (VB == 4) {
          float2 v = make_float2(fmaf(r0, one, zs[m >> 1][k]), fmaf(r1, one * 0.0625f, zs[m >> 1][k]));
          *reinterpret_cast<float2*>(dst + 16 * m + 2 * g) = v;
        } else {
          const float s0 = (m & 1) ? one * 0.0625f : one, s1 = (m & 1) ? one * 0.015625f : one * 0.25f;
          float2 v = make_float2(fmaf(r0, s0, zs[m >> 1][k]), fmaf(r1, s1, zs[m >> 1][k]));
          *reinterpret_cast<float2*>(dst + 32 * (m >> 1) + 4 * g + 2 * (m & 1)) = v;
        }
      }
    }
  };

  int sk = 0, sv = 0, pk = 0, pv = 0;  // ring slots and their phases
  int j = 0;
  bool landed = true;  // every copy so far
#pragma unroll 1
  while (landed) {  // segments; the query's words are live between them only
    prepare_query(unit, tiles[j & 63].msk, raw0);
#pragma unroll 1
    do {
      if ((j & 31) == 16) look_up((j >> 5) + 1);  // the issue runs at most 4 tiles ahead
      const int nval = tiles[j & 63].nval;
      if (!(landed = wait_full(kbars + 8 * sk, pk))) break;
      float p[4][2][HT];  // the scores, then 2^(score - M), of tokens 8g + 2i + e
      if (nval > 0) {
        const uint8_t* st = kring + sk * S::KPART;
        // ================================================================ scores
        float acc[4][NA][4];
        {
          const uint4 z0 = *reinterpret_cast<const uint4*>(st + S::K_ZEROS + (g * 2 + (cq & 1)) * 16);
          const uint4 z1 = *reinterpret_cast<const uint4*>(st + S::K_ZEROS + ((8 + g) * 2 + (cq & 1)) * 16);
#pragma unroll
          for (int na = 0; na < NA; ++na) {
            const uint32_t bz = qz[na * 32 + lane], bl = HC == 4 ? 0 : qz[((NT - NA) + na) * 32 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4& z = i < 2 ? z0 : z1;
              mma8z(acc[i][na], (i & 1) ? z.z : z.x, (i & 1) ? z.w : z.y, bz);
              if (HC > 4) mma8(acc[i][na], (i & 1) ? z.z : z.x, (i & 1) ? z.w : z.y, bl);
            }
          }
        }
        uint4 ks[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = *reinterpret_cast<const uint4*>(st + S::K_SCALES + 16 * (8 * i + g));
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
            uint32_t ka[8];
            if (KB == 4 && !PREC) {
              // a token's byte whole (code + 16 code'), and its upper field: the query is
              // given in that basis
              ka[0] = __byte_perm(word(w0, i), 0, 0x4240);
              ka[1] = __byte_perm(word(w0, i), 0, 0x4341);
              ka[2] = ka[0] & 0x00F000F0u;
              ka[3] = ka[1] & 0x00F000F0u;
              ka[4] = __byte_perm(word(w1, i), 0, 0x4240);
              ka[5] = __byte_perm(word(w1, i), 0, 0x4341);
              ka[6] = ka[4] & 0x00F000F0u;
              ka[7] = ka[5] & 0x00F000F0u;
            } else {
              const uint32_t x = word(w0, i), y = KB == 4 ? word(w1, i) : x;
              const uint32_t xs = x >> 8, ys = KB == 4 ? y >> 8 : xs;
              constexpr uint32_t m0 = KB == 4 ? 0x000F000Fu : 0x00030003u, m1 = KB == 4 ? 0x00F000F0u : 0x000C000Cu;
              constexpr uint32_t m2 = KB == 4 ? m0 : 0x00300030u, m3 = KB == 4 ? m1 : 0x00C000C0u;
              ka[0] = codes_of<PREC>(x, m0, 0);
              ka[1] = codes_of<PREC>(xs, m0, 0);
              ka[2] = codes_of<PREC>(x, m1, 0);
              ka[3] = codes_of<PREC>(xs, m1, 0);
              ka[4] = codes_of<PREC>(y, m2, 0);
              ka[5] = codes_of<PREC>(ys, m2, 0);
              ka[6] = codes_of<PREC>(y, m3, 0);
              ka[7] = codes_of<PREC>(ys, m3, 0);
            }
            const float2 sa = float2_of((Q >> 1) ? ks[i].y : ks[i].x), sb = float2_of((Q >> 1) ? ks[i].w : ks[i].z);
            const float s0 = (Q & 1) ? sa.y : sa.x, s1 = (Q & 1) ? sb.y : sb.x;
#pragma unroll
            for (int na = 0; na < NA; ++na) {
              float d[4];
              mma16z(d, ka[0], ka[1], ka[2], ka[3], bA[NT - NA + na].x, bA[NT - NA + na].y);
              mma16(d, ka[4], ka[5], ka[6], ka[7], bB[NT - NA + na].x, bB[NT - NA + na].y);
              if (HC > 4) {  // the low pieces came first
                mma16(d, ka[0], ka[1], ka[2], ka[3], bA[na].x, bA[na].y);
                mma16(d, ka[4], ka[5], ka[6], ka[7], bB[na].x, bB[na].y);
              }
              acc[i][na][0] = fmaf(s0, d[0], acc[i][na][0]);
              acc[i][na][1] = fmaf(s0, d[1], acc[i][na][1]);
              acc[i][na][2] = fmaf(s1, d[2], acc[i][na][2]);
              acc[i][na][3] = fmaf(s1, d[3], acc[i][na][3]);
            }
          }
        }
        float q0[HT] = {};
        if (CH0) {
#pragma unroll
          for (int k = 0; k < HT; ++k) q0[k] = qh[head_of(k)].y;
        }
        uint4 k0 = make_uint4(0, 0, 0, 0);
        if (CH0) k0 = *reinterpret_cast<const uint4*>(st + S::K_CH0 + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t kk = word(k0, i);
            const float kv = __uint_as_float(e ? kk & 0xFFFF0000u : kk << 16);
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              float sc = HC == 4 ? fmaf(acc[i][0][2 * e + 1], kLow, acc[i][0][2 * e]) : acc[i][k >> 1][2 * e + (k & 1)];
              if (CH0) sc = fmaf(q0[k], kv, sc);
              p[i][e][k] = sc;
            }
          }
        if (nval < kBlockTokens) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < HT; ++k)
                if (8 * g + 2 * i + e >= nval) p[i][e][k] = qh[head_of(k)].x < 0.0f ? INFINITY : -INFINITY;
        }
      }
      __syncwarp();  // every lane has read the slot
      if (j + SK < n) issue_keys(j + SK, sk);
      if (++sk == SK) {
        sk = 0;
        pk ^= 1;
      }
      if (!(landed = wait_full(vbars + 8 * sv, pv))) break;
      if (nval > 0) {
        uint8_t* st = vring + sv * S::VPART;
        if (nval < kBlockTokens) {  // bytes behind the last token may hold anything: no scale, no zero there
#pragma unroll
          for (int t = lane; t < kBlockTokens; t += 32)
            if (t >= nval) {
              *reinterpret_cast<uint2*>(st + S::V_SCALES + 2 * scale_index(t, 0)) = make_uint2(0, 0);
              *reinterpret_cast<uint2*>(st + S::V_ZEROS + 2 * scale_index(t, 0)) = make_uint2(0, 0);
            }
          fence_proxy_async();  // before a later copy into this slot
          __syncwarp();
        }
        uint4 vs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) vs[i] = *reinterpret_cast<const uint4*>(st + S::V_SCALES + 16 * (8 * i + g));
        // ================================================================ softmax
        // p = 2^(s - M) against bounds: p <= plim keeps p and p * scale below 2^15.
        // Lane (g, cq) checks the scales of two of its row's tokens.
        float tile_scale;
        {
          const uint4 v = *reinterpret_cast<const uint4*>(st + S::V_SCALES + 16 * (8 * cq + g));
          const float2 m = float2_of(hmax2(hmax2(v.x, v.y), hmax2(v.z, v.w)));
          tile_scale = fmaxf(m.x, m.y);
        }
        bool over = tile_scale > smax;
        float x[4][2][HT], fac[HT];  // fac: score units to log2
#pragma unroll
        for (int k = 0; k < HT; ++k) fac[k] = qh[head_of(k)].x;
#pragma unroll
        for (int k = 0; k < HT; ++k) {
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i][0][k] = ex2(fmaf(p[i][0][k], fac[k], -M[k]));
            x[i][1][k] = ex2(fmaf(p[i][1][k], fac[k], -M[k]));
            top = fmaxf(top, fmaxf(x[i][0][k], x[i][1][k]));
          }
          over |= top > plim;
        }
        if (__any_sync(kFull, over)) {
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) tile_scale = fmaxf(tile_scale, __shfl_xor_sync(kFull, tile_scale, m));
          float turn = 1.0f;  // of the sums so far, to the new power
          if (tile_scale > smax) {
            smax = 1.25f * tile_scale;  // the next largest ones do not come back here
            const float next = scales_up(smax);
            turn = __int_as_float(__float_as_int(next) - __float_as_int(up) + (127 << 23));
            up = next;
          }
          plim = kTop16 / fmaxf(smax * up, 1.0f);
          // the largest p becomes plim / 2^8 (the room for later ones), but 2^6 where it can
          const float room = fmaxf(__log2f(plim) - 8.0f, fminf(__log2f(plim) - 1.0f, 6.0f));
#pragma unroll
          for (int k = 0; k < HT; ++k) {
            float t = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) t = fmaxf(t, fmaxf(p[i][0][k] * fac[k], p[i][1][k] * fac[k]));
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) t = fmaxf(t, __shfl_xor_sync(kFull, t, m));
            const float m_new = fmaxf(M[k], t - room);
            const float al = ex2(M[k] - m_new);
            M[k] = m_new;
            l[k] *= al;
            if (PREC) {
#pragma unroll
              for (int r = 0; r < kGroups; ++r) zs[r][k] *= al;
            } else {
              zp[k >> 1][k & 1] *= al;
              zp[k >> 1][2 + (k & 1)] *= al;
            }
            const float ao = al * turn;
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              if (HC == 4) {
                O[m][0] *= ao;
                O[m][1] *= ao;
              } else {
                O[m][4 * (k >> 1) + (k & 1)] *= ao;
                O[m][4 * (k >> 1) + 2 + (k & 1)] *= ao;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) x[i][e][k] = ex2(fmaf(p[i][e][k], fac[k], -m_new));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int k = 0; k < HT; ++k) {
              p[i][e][k] = x[i][e][k];
              if (PREC) l[k] += x[i][e][k];
            }
        constexpr int kMid = S::MID;
        uint32_t ph[4][2][NH];  // p as fp16: the head twice (HC = 4), or a pair of heads
        if (!PREC) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int t = 0; t < NH; ++t)
                ph[i][e][t] = HC == 4 ? half2_of(p[i][e][0], p[i][e][0]) : half2_of(p[i][e][(2 * t) % HT], p[i][e][(2 * t + 1) % HT]);
          // zero-point sums: matrix i's transposed rows are (e, group), its columns the
          // tokens 8u + 2i + e; rows 0-3 meet the even tokens in the lower half of K,
          // rows 12-15 the odd ones in the upper half, the others are not used
          const uint4 z = load_transposed(smem_addr(st + S::V_ZEROS + 16 * lane));
          // kF16 counts codes from their middle, and the middle times the scale may pass fp16
          // where value and output do not (rotated values): the scales' sums are rows of their
          // own, in the places that are free: 4-7 the odd tokens', 8-11 the even ones'
          const uint4 vt = MODE == kF16 ? load_transposed(smem_addr(st + S::V_SCALES + 16 * lane)) : make_uint4(0, 0, 0, 0);
          constexpr uint32_t kOnes = 0x3C003C00u;
          auto add_zeros = [&](float (&d)[4], int i, uint32_t b0, uint32_t b1) {
            const uint32_t zi = word(z, i), si = word(vt, i);
            if (MODE == kF16)
              mma16(d, g < 4 ? zi : 0u, g < 4 ? si : 0u, g < 4 ? 0u : si, g < 4 ? 0u : zi, b0, b1);
            else if (S::ONES)
              mma16(d, zi, 0u, 0u, zi, b0, b1);
            else  // row 4 sums the rounded p
              mma16(d, g == 4 ? kOnes : zi, 0u, g == 4 ? kOnes : 0u, zi, b0, b1);
          };
#pragma unroll
          for (int t = 0; t < NH; ++t) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dl[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b0 = transpose8(ph[i][0][t]), b1 = transpose8(ph[i][1][t]);
              add_zeros(d, i, b0, b1);
              if (S::ONES) mma16(dl, kOnes, kOnes, kOnes, kOnes, b0, b1);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) zp[t][r] += d[r];
            if (S::ONES) {  // the same in all rows
              l[(2 * t) % HT] += dl[0];
              if (HC > 4) l[(2 * t + 1) % HT] += dl[1];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 vz = *reinterpret_cast<const uint4*>(st + S::V_ZEROS + 16 * (8 * i + g));
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float2 z = float2_of(word(vz, 2 * e + r)), sv = float2_of(word(vs[i], 2 * e + r));
                const float za = fmaf((float)kMid, sv.x, z.x), zb = fmaf((float)kMid, sv.y, z.y);
#pragma unroll
                for (int k = 0; k < HT; ++k) {
                  zs[2 * r][k] = fmaf(p[i][e][k], za, zs[2 * r][k]);
                  zs[2 * r + 1][k] = fmaf(p[i][e][k], zb, zs[2 * r + 1][k]);
                }
              }
          }
        }
        // ================================================================ value sums
        if (up != 1.0f) {  // the same in all lanes
          if (PREC) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < HT; ++k) p[i][e][k] *= up;
          } else {  // in two steps: the power itself may be outside fp16
            const int ex = (__float_as_int(up) >> 23) - 127;
            const float u0 = __int_as_float((127 + (ex >> 1)) << 23), u1 = __int_as_float((127 + ex - (ex >> 1)) << 23);
            const uint32_t h0 = half2_of(u0, u0), h1 = half2_of(u1, u1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              vs[i].x = hmul2(hmul2(vs[i].x, h0), h1);
              vs[i].y = hmul2(hmul2(vs[i].y, h0), h1);
              vs[i].z = hmul2(hmul2(vs[i].z, h0), h1);
              vs[i].w = hmul2(hmul2(vs[i].w, h0), h1);
            }
          }
        }
        constexpr int NR = S::PAIR ? 2 : 4;  // rounds: a pair of groups or one group each
#pragma unroll
        for (int rd = 0; rd < NR; ++rd) {
          uint32_t b[4][NP][2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (S::PAIR) {
                b[i][0][e] = transpose8(hmul2(ph[i][e][0], word(vs[i], 2 * e + rd)));
              } else if (!PREC) {
                const uint32_t sv = dup_half(word(vs[i], 2 * e + (rd >> 1)), rd & 1);
#pragma unroll
                for (int t = 0; t < NH; ++t) b[i][t][e] = transpose8(hmul2(ph[i][e][t], sv));
              } else {
                const float2 s2 = float2_of(word(vs[i], 2 * e + (rd >> 1)));
                const float sv = (rd & 1) ? s2.y : s2.x;
                if (HC == 4) {
                  const float v = p[i][e][0] * sv;
                  const float hi = __half2float(__float2half_rn(v));
                  b[i][0][e] = transpose8(half2_of(hi, (v - hi) * 2048.0f));
                } else {
#pragma unroll
                  for (int t = 0; t < NH; ++t) {
                    const float v0 = p[i][e][(2 * t) % HT] * sv, v1 = p[i][e][(2 * t + 1) % HT] * sv;
                    const uint32_t hi = half2_of(v0, v1);
                    const float2 f = float2_of(hi);
                    b[i][t][e] = transpose8(hi);
                    b[i][(NP / 2 + t) % NP][e] = transpose8(half2_of((v0 - f.x) * 2048.0f, (v1 - f.y) * 2048.0f));
                  }
                }
              }
            }
          // minus the codes' middle times the sum of the rounded P' (all rows alike)
          float base[NP][4];
          if (MODE == kF16) {
            constexpr uint32_t c0 = VB == 4 ? 0x80088008u : 0x80028002u, c1 = VB == 4 ? 0x80808080u : 0x80088008u;
#pragma unroll
            for (int np = 0; np < NP; ++np) {
              mma16z(base[np], c0, c1, c0, c1, b[0][np][0], b[0][np][1]);
#pragma unroll
              for (int i = 1; i < 4; ++i) mma16(base[np], c0, c1, c0, c1, b[i][np][0], b[i][np][1]);
            }
          }
          constexpr int MT = S::PAIR ? 4 : 2;  // 16-channel tiles of this round
#pragma unroll
          for (int mm = 0; mm < MT; ++mm) {
            const int m = rd * MT + mm;
            const uint4 w = *reinterpret_cast<const uint4*>(st + ((VB == 4 ? m : m >> 1) * 8 + g) * 64 + cq * 16);
            const uint32_t m0 = VB == 4 ? 0x000F000Fu : (m & 1) ? 0x00300030u : 0x00030003u;
            const uint32_t m1 = VB == 4 ? 0x00F000F0u : (m & 1) ? 0x00C000C0u : 0x000C000Cu;
            float d[NP][4];
            if (MODE == kF16) {
#pragma unroll
              for (int np = 0; np < NP; ++np)
#pragma unroll
                for (int r = 0; r < 4; ++r) d[np][r] = (VB == 2 && (m & 1)) ? 16.0f * base[np][r] : base[np][r];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = word(w, i), xs = x >> 8;
              constexpr int f1 = VB == 4 ? 16 : 4;  // the fields' factors
              const int f = VB == 4 ? 1 : (m & 1) ? 16 : 1;
              const uint32_t a0 = codes_of<PREC>(x, m0, f * kMid), a1 = codes_of<PREC>(x, m1, f * f1 * kMid);
              const uint32_t a2 = codes_of<PREC>(xs, m0, f * kMid), a3 = codes_of<PREC>(xs, m1, f * f1 * kMid);
#pragma unroll
              for (int np = 0; np < NP; ++np) {
                if (i == 0 && MODE != kF16)
                  mma16z(d[np], a0, a1, a2, a3, b[i][np][0], b[i][np][1]);
                else
                  mma16(d[np], a0, a1, a2, a3, b[i][np][0], b[i][np][1]);
              }
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
              for (int t = 0; t < NH; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  O[m][4 * t + r] += PREC ? fmaf(d[(NP / 2 + t) % NP][r], kLow, d[t][r]) : d[t][r];
            }
          }
        }
      }
      __syncwarp();  // every lane has read the slot
      if (j + SV < n) issue_values(j + SV, sv);
      if (++sv == SV) {
        sv = 0;
        pv ^= 1;
      }
      ++j;
    } while (j < n && tiles[j & 63].unit == unit);
    if (!landed) break;
    end_segment();
    if (j == n) break;
    unit = tiles[j & 63].unit;
    load_query(unit, raw0);
  }
  if (__builtin_expect(!landed, 0)) {
    // a copy did not land in time: not-a-number partials for this segment and the
    // rest of the range, and time for copies in flight to land before the
    // shared memory is given up
    int last = -1;
    for (int x = j; x < n; ++x) {
      if (x != j && (x & 31) == 16) look_up((x >> 5) + 1);
      const int u = tiles[x & 63].unit;
      if (u == last) continue;
      last = u;
      const size_t row = (size_t)(u + rank) * a.G + lane;
      if (lane < a.G && kvq_in_bounds(row, 1, a.part_rows)) a.part_ml[row] = make_float2(NAN, NAN);
    }
    __nanosleep(64000);
  }
  if (lane == 0) a.status[rank] = landed ? 0 : 1;
  let_next_start();
}

template <int KB, int VB, int HC, int MODE, bool CH0>
cudaError_t launch_one(const PagedDecodeArgs& a, cudaStream_t s) {
  using S = Shape<KB, VB, HC, MODE, CH0>;
  auto kern = k_paged_decode<KB, VB, HC, MODE, CH0>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may take this much shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_overlapped(kern, dim3(kSms), dim3(S::THREADS), S::SMEM, s, a);
}

template <int KB, int VB, int HC, int MODE>
cudaError_t launch_ch0(const PagedDecodeArgs& a, cudaStream_t s) {
  return a.c.keep_ch0 ? launch_one<KB, VB, HC, MODE, true>(a, s) : launch_one<KB, VB, HC, MODE, false>(a, s);
}

template <int KB, int VB, int HC>
cudaError_t launch_type(const PagedDecodeArgs& a, cudaStream_t s) {
  if (a.dtype == KVQ_F32) return launch_ch0<KB, VB, HC, kF32>(a, s);
  return a.dtype == KVQ_F16 ? launch_ch0<KB, VB, HC, kF16>(a, s) : launch_ch0<KB, VB, HC, kBf16>(a, s);
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
