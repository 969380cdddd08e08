// Joining the paged decode's partials: one softmax per (request, query head).
#include "paged_decode.cuh"

namespace kvq {
namespace paged {
namespace {

__device__ __forceinline__ void store4(void* out, int dtype, size_t at, const float (&x)[4]) {
  if (dtype == KVQ_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(x[0], x[1], x[2], x[3]);
  } else if (dtype == KVQ_BF16) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<uint2*>(static_cast<__half*>(out) + at) = make_uint2(half2_of(x[0], x[1]), half2_of(x[2], x[3]));
  }
}

// WPR warps per output row, lane = 4 channels.  A row's partials sit in slots
// unit + r of the ranks r its tiles touch, as the split cut them.
template <int WPR>
__global__ void __launch_bounds__(256) k_paged_combine(PagedDecodeArgs a, int max_ranks) {
  __shared__ float2 sml[8];
  __shared__ float4 sacc[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * (8 / WPR) + warp / WPR;
  const int part = warp % WPR;
  const bool live = row < a.B * a.Hq;
  let_next_start();
  wait_for_stream();  // the split decode's partials are complete
  float m = -INFINITY, l = 0.0f;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (live) {
    const int b = row / a.Hq, j = row - b * a.Hq, H = a.c.H, h = j / a.G, hd = j - h * a.G;
    const int total = a.starts[a.B] * H;
    const int s0 = a.starts[b], tiles = a.starts[b + 1] - s0;
    if (tiles > 0) {
      const int ranks = min(max_ranks, total), x = s0 * H + h * tiles;
      const int r0 = rank_of(x, ranks, total), r1 = rank_of(x + tiles - 1, ranks, total);
      const size_t unit = (size_t)b * H + h;
      constexpr int U = WPR == 1 ? 2 : 8;  // partials in flight per warp
      for (int r = r0 + part; r <= r1; r += U * WPR) {
        float2 ml[U];
        float4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int rr = r + k * WPR;
          ml[k] = make_float2(-INFINITY, 0.0f);
          v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const size_t pr = (unit + rr) * a.G + hd;
          if (rr <= r1 && kvq_in_bounds(pr, 1, a.part_rows)) {
            ml[k] = a.part_ml[pr];
            v[k] = *reinterpret_cast<const float4*>(a.part_acc + pr * kHeadDim + 4 * lane);
          }
        }
        float mn = m;
#pragma unroll
        for (int k = 0; k < U; ++k) mn = fmaxf(mn, ml[k].x);
        const float al = m == mn ? 1.0f : exp2f(m - mn);
        l *= al;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= al;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float w = ml[k].x == -INFINITY ? 0.0f : exp2f(ml[k].x - mn);
          l = fmaf(w, ml[k].y, l);
          acc[0] = fmaf(w, v[k].x, acc[0]);
          acc[1] = fmaf(w, v[k].y, acc[1]);
          acc[2] = fmaf(w, v[k].z, acc[2]);
          acc[3] = fmaf(w, v[k].w, acc[3]);
        }
        m = mn;
      }
    }
  }
  if (WPR > 1) {
    if (lane == 0) sml[warp] = make_float2(m, l);
    sacc[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (part != 0) return;
    float mn = m;
#pragma unroll
    for (int k = 1; k < WPR; ++k) mn = fmaxf(mn, sml[warp + k].x);
    const float al = m == mn ? 1.0f : exp2f(m - mn);
    l *= al;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= al;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float2 o = sml[warp + k];
      const float w = o.x == -INFINITY ? 0.0f : exp2f(o.x - mn);
      const float4 v = sacc[warp + k][lane];
      l = fmaf(w, o.y, l);
      acc[0] = fmaf(w, v.x, acc[0]);
      acc[1] = fmaf(w, v.y, acc[1]);
      acc[2] = fmaf(w, v.z, acc[2]);
      acc[3] = fmaf(w, v.w, acc[3]);
    }
  }
  if (!live) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no token took part: a zero row
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] *= inv;
  if (a.c.rotate_v) {
    const float y0 = acc[0] + acc[1], y1 = acc[0] - acc[1], y2 = acc[2] + acc[3], y3 = acc[2] - acc[3];
    acc[0] = y0 + y2;
    acc[1] = y1 + y3;
    acc[2] = y0 - y2;
    acc[3] = y1 - y3;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const float sg = (lane & k) ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(sg, acc[i], __shfl_xor_sync(kFull, acc[i], k));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= 0.08838834764831845f;
  }
  store4(a.out, a.dtype, (size_t)row * kHeadDim + 4 * lane, acc);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t s) {
  using namespace paged;
  cudaError_t e = a.c.k_bits == 4 ? (a.c.v_bits == 4 ? launch_44(a, s) : launch_42(a, s))
                                  : (a.c.v_bits == 4 ? launch_24(a, s) : launch_22(a, s));
  if (e != cudaSuccess) return e;
  const int ranks = paged_decode_ranks(a.G, a.dtype);
  // one warp per row where a row has few partials, a block per row where its
  // sequence was cut into many
  const long long units = (long long)a.B * a.c.H, rows = (long long)a.B * a.Hq;
  const bool many = ranks / units >= 8;
  if (many) return launch_overlapped(k_paged_combine<8>, dim3((unsigned)rows), dim3(256), 0, s, a, ranks);
  return launch_overlapped(k_paged_combine<1>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a, ranks);
}

unsigned bounds_paged_decode(bool reset) {
  return paged::bounds_44(reset) + paged::bounds_42(reset) + paged::bounds_24(reset) + paged::bounds_22(reset);
}

}  // namespace kvq
