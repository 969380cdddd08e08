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

// A warp's sums over the partials of (unit, head hd) left by ranks r, r + step, ...
// up to r1, U in flight at a time; lane = channels 4 lane .. 4 lane + 3
struct Joined {
  float m, l, acc[4];
};
template <int U>
__device__ __forceinline__ void join_partials(const PagedDecodeArgs& a, size_t unit, int hd, int r, int r1, int step, int lane,
                                              Joined& s) {
  s.m = -INFINITY;
  s.l = s.acc[0] = s.acc[1] = s.acc[2] = s.acc[3] = 0.0f;
#pragma unroll 1
  for (; r <= r1; r += U * step) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int rr = r + k * step;
      ml[k] = make_float2(-INFINITY, 0.0f);
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const size_t pr = (unit + rr) * a.G + hd;
      if (rr <= r1 && kvq_in_bounds(pr, 1, a.part_rows)) {
        ml[k] = __ldcg(a.part_ml + pr);
        v[k] = __ldcg(reinterpret_cast<const float4*>(a.part_acc + pr * kHeadDim + 4 * lane));
      }
    }
    float mn = s.m;
#pragma unroll
    for (int k = 0; k < U; ++k) mn = fmaxf(mn, ml[k].x);
    const float al = s.m == mn ? 1.0f : exp2f(s.m - mn);
    s.l *= al;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.acc[i] *= al;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float w = ml[k].x == -INFINITY ? 0.0f : exp2f(ml[k].x - mn);
      s.l = fmaf(w, ml[k].y, s.l);
      s.acc[0] = fmaf(w, v[k].x, s.acc[0]);
      s.acc[1] = fmaf(w, v[k].y, s.acc[1]);
      s.acc[2] = fmaf(w, v[k].z, s.acc[2]);
      s.acc[3] = fmaf(w, v[k].w, s.acc[3]);
    }
    s.m = mn;
  }
}
// ... divided, taken back through the value rotation, rounded and written
__device__ __forceinline__ void finish_row(const PagedDecodeArgs& a, size_t row, int lane, Joined& s) {
  const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;  // no token took part: a zero row
  float(&x)[4] = s.acc;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] *= inv;
  if (a.c.rotate_v) {
    const float y0 = x[0] + x[1], y1 = x[0] - x[1], y2 = x[2] + x[3], y3 = x[2] - x[3];
    x[0] = y0 + y2;
    x[1] = y1 + y3;
    x[2] = y0 - y2;
    x[3] = y1 - y3;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const float sg = (lane & k) ? -1.0f : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmaf(sg, x[i], __shfl_xor_sync(kFull, x[i], k));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= 0.08838834764831845f;  // 1 / sqrt(128)
  }
  store4(a.out, a.dtype, row * kHeadDim + 4 * lane, x);
}

// WPR warps per output row: one where a row has few partials (a block then takes
// eight rows), eight where its sequence was cut into many: 16 ranks a unit or more
// (us of the whole decode with one and eight: 296 units of 8 ranks 39 and 44; 128 of 18
// 22.2 and 22.0; 64 of 37 67.8 and 62.8; 8 of 296 64 and 24).  The rule goes by the
// average: one request of 128K tokens among 63 of 256 takes 76 us, one warp joining each of
// the long request's rows of some 270 partials.  A row's partials sit
// in slots unit + r of the ranks r its tiles touch, as the split cut them.
template <int WPR>
__global__ void __launch_bounds__(256) k_paged_join(PagedDecodeArgs a, int max_ranks) {
  __shared__ float2 sml[8];
  __shared__ float4 sacc[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * (8 / WPR) + warp / WPR;
  const bool live = row < a.B * a.Hq;
  let_next_start();
  wait_for_stream();  // the split decode's partials are complete
  Joined s;
  s.m = -INFINITY;
  s.l = s.acc[0] = s.acc[1] = s.acc[2] = s.acc[3] = 0.0f;
  if (live) {
    const int b = row / a.Hq, j = row - b * a.Hq, H = a.c.H, h = j / a.G, hd = j - h * a.G;
    const int total = a.starts[a.B] * H, s0 = a.starts[b], tiles = a.starts[b + 1] - s0;
    if (tiles > 0) {
      const int ranks = min(max_ranks, total), x = s0 * H + h * tiles;
      const int r0 = rank_of(x, ranks, total), r1 = rank_of(x + tiles - 1, ranks, total);
      join_partials<WPR == 1 ? 4 : 8>(a, (size_t)b * H + h, hd, r0 + warp % WPR, r1, WPR, lane, s);
    }
  }
  if (WPR > 1) {
    if (lane == 0) sml[warp] = make_float2(s.m, s.l);
    sacc[warp][lane] = make_float4(s.acc[0], s.acc[1], s.acc[2], s.acc[3]);
    __syncthreads();
    if (warp != 0) return;
    float mn = s.m;
#pragma unroll
    for (int k = 1; k < 8; ++k) mn = fmaxf(mn, sml[k].x);
    const float al = s.m == mn ? 1.0f : exp2f(s.m - mn);
    s.l *= al;
#pragma unroll
    for (int i = 0; i < 4; ++i) s.acc[i] *= al;
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      const float2 o = sml[k];
      const float w = o.x == -INFINITY && o.y == 0.0f ? 0.0f : exp2f(o.x - mn);  // not-a-number sums stay in
      const float4 v = sacc[k][lane];
      s.l = fmaf(w, o.y, s.l);
      s.acc[0] = fmaf(w, v.x, s.acc[0]);
      s.acc[1] = fmaf(w, v.y, s.acc[1]);
      s.acc[2] = fmaf(w, v.z, s.acc[2]);
      s.acc[3] = fmaf(w, v.w, s.acc[3]);
    }
  }
  if (live) finish_row(a, row, lane, s);
}

}  // namespace
}  // namespace paged

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, cudaStream_t s) {
  using namespace paged;
  cudaError_t e = a.c.k_bits == 4 ? (a.c.v_bits == 4 ? launch_44(a, s) : launch_42(a, s))
                                  : (a.c.v_bits == 4 ? launch_24(a, s) : launch_22(a, s));
  if (e != cudaSuccess) return e;
  const int ranks = paged_decode_ranks(a.G, a.dtype), rows = a.B * a.Hq;
  if (ranks / ((long long)a.B * a.c.H) >= 16) return launch_overlapped(k_paged_join<8>, dim3(rows), dim3(256), 0, s, a, ranks);
  return launch_overlapped(k_paged_join<1>, dim3((rows + 7) / 8), dim3(256), 0, s, a, ranks);
}

unsigned bounds_paged_decode(bool reset) {
  return paged::bounds_44(reset) + paged::bounds_42(reset) + paged::bounds_24(reset) + paged::bounds_22(reset);
}

}  // namespace kvq
