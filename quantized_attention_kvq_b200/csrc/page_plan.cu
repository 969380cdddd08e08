// One scheduling step's block tables and slot map, in one launch.
//
// Three prefix sums over the requests carry everything: new tokens (the flat
// token list), pages needed (places on the free stack) and pages given back
// (places the finished requests push to).  The j-th page of the step is
// free_pages[top - 1 - j], top = count + pages given back, so which request gets
// which page is known to every thread from the sums alone.
//
// Latency-bound: a step touches a few KB to a few MB.  One cluster of CTAs (one
// CTA for a small step) shares the work; every CTA makes the three sums for
// itself in shared memory (cheaper than passing them on), pushes its share of
// the returned pages, meets the others at the cluster barrier, and then fills
// its share of the table entries and slots, each found by a binary search in
// the sums.  The barrier also separates reading *free_count, ctx_lens and the
// finished requests' table rows from writing them, so they may be updated in
// place.
// Measured on B200, launched back to back in a graph: 5.1 us for 8 requests (nothing
// but latencies in a row), 12.2 us for 512 requests of which 48 bring 120,000 new
// tokens, 21.8 us for 512,000 (4 MB written).
#include <atomic>

#include <cooperative_groups.h>

#include "paged.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kPortable = 8, kWidest = 16;  // CTAs of a cluster

// last b with sum[b] <= x, for 0 <= x < sum[n]
__device__ __forceinline__ int find(const int* sum, int n, int x) {
  int lo = 0, hi = n;  // sum[lo] <= x < sum[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (sum[m] <= x)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

__device__ __forceinline__ int pages_for(int tokens, const Divisor& P) {
  const int q = P.quotient(tokens);
  return q + ((uint32_t)q * P.d != (uint32_t)tokens);
}

template <int TH>
__global__ void __launch_bounds__(TH) k_page_plan(PlanArgs a) {
  extern __shared__ int sm[];
  const int B = a.batch, P = a.page_tokens, tid = threadIdx.x;
  int* cu = sm;                 // [B + 1] new tokens before request b
  int* need = cu + B + 1;       // [B + 1] pages needed before request b
  int* give = need + B + 1;     // [B + 1] pages given back before request b
  int* ctx = give + B + 1;      // [B] cached tokens, 0 for finished requests
  __shared__ long long wsum[2][TH / 32];
  __shared__ int taken_s;
  let_next_start();
  wait_for_stream();
  const int count = min(max(*a.count, 0), a.num_pages);

  // each thread sums a run of consecutive requests; the runs are joined by a
  // scan over the threads.  Sums are 64-bit and saturate when stored.
  const int per = (B + TH - 1) / TH;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  const int first_ctx = b0 < b1 ? a.ctx[b0] : 0, first_add = b0 < b1 ? a.add[b0] : 0;  // the only one, as a rule
  const bool first_fin = b0 < b1 && a.done && a.done[b0] != 0;
  auto ctx_of = [&](int b) { return max(b == b0 ? first_ctx : a.ctx[b], 0); };
  auto add_of = [&](int b) { return max(b == b0 ? first_add : a.add[b], 0); };
  auto finished = [&](int b) { return b == b0 ? first_fin : a.done && a.done[b] != 0; };
  constexpr long long kMax = 0x7FFFFFFF;
  long long s[2] = {0, 0};
  const long long row_tokens = (long long)a.max_pages * P;
  // pass 0: new tokens and pages given back; pass 1: pages needed, which depend on cu
  for (int pass = 0; pass < 2; ++pass) {
    long long t0 = 0, t1 = 0;
    for (int b = b0; b < b1; ++b) {
      if (pass == 0) {
        const bool fin = finished(b);
        const int c = ctx_of(b);
        t0 += add_of(b);
        t1 += fin ? min(pages_for(c, a.page), a.max_pages) : 0;
        ctx[b] = fin ? 0 : c;
      } else {
        const long long end = (long long)ctx[b] + add_of(b);
        const bool fits = end <= row_tokens && cu[b + 1] <= a.n_slots;
        t0 += fits ? pages_for((int)end, a.page) - pages_for(ctx[b], a.page) : 0;
      }
    }
    long long x0 = t0, x1 = t1;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long y0 = __shfl_up_sync(kFull, x0, m), y1 = __shfl_up_sync(kFull, x1, m);
      if ((tid & 31) >= m) {
        x0 += y0;
        x1 += y1;
      }
    }
    if ((tid & 31) == 31) {
      wsum[0][tid >> 5] = x0;
      wsum[1][tid >> 5] = x1;
    }
    __syncthreads();
    // every warp scans the warps' totals for itself
    constexpr int NW = TH / 32;
    static_assert(NW <= 32, "one total per lane");
    long long y0 = wsum[0][tid & (NW - 1)], y1 = wsum[1][tid & (NW - 1)];
#pragma unroll
    for (int m = 1; m < NW; m <<= 1) {
      const long long z0 = __shfl_up_sync(kFull, y0, m), z1 = __shfl_up_sync(kFull, y1, m);
      if ((tid & 31) >= m) {
        y0 += z0;
        y1 += z1;
      }
    }
    const int prev = (tid >> 5) - 1;
    y0 = __shfl_sync(kFull, y0, prev & 31);
    y1 = __shfl_sync(kFull, y1, prev & 31);
    s[0] = x0 - t0 + (prev >= 0 ? y0 : 0);
    s[1] = x1 - t1 + (prev >= 0 ? y1 : 0);
    int* out0 = pass == 0 ? cu : need;
    if (tid == 0) {
      out0[0] = 0;
      if (pass == 0) give[0] = 0;
      taken_s = 0;
    }
    for (int b = b0; b < b1; ++b) {
      if (pass == 0) {
        s[0] += add_of(b);
        s[1] += finished(b) ? min(pages_for(ctx_of(b), a.page), a.max_pages) : 0;
        cu[b + 1] = (int)min(s[0], kMax);
        give[b + 1] = (int)min(s[1], kMax);
      } else {
        const long long end = (long long)ctx[b] + add_of(b);
        const bool fits = end <= row_tokens && cu[b + 1] <= a.n_slots;
        s[0] += fits ? pages_for((int)end, a.page) - pages_for(ctx[b], a.page) : 0;
        need[b + 1] = (int)min(s[0], kMax);
      }
    }
    __syncthreads();
  }
  const int returned = give[B];
  const int top = (int)min((long long)count + returned, (long long)a.num_pages);

  // pages taken: the largest prefix of needed pages that the stack covers
  int mine = 0;
  for (int b = b0; b < b1; ++b)
    if (need[b + 1] <= top) mine = max(mine, need[b + 1]);
  mine = __reduce_max_sync(kFull, mine);
  if ((tid & 31) == 0) atomicMax(&taken_s, mine);

  const int gt = blockIdx.x * TH + tid, gn = gridDim.x * TH;
  for (int r = gt; r < top - count; r += gn) {  // all of them, unless lengths were wrong and the stack is full
    const int b = find(give, B, r);
    a.free_pages[count + r] = a.table[(size_t)b * a.max_pages + (r - give[b])];
  }
  if (gridDim.x > 1)
    cg::this_cluster().sync();  // pushed pages visible; every CTA has read what is updated in place
  else
    __syncthreads();
  const int taken = taken_s;

  for (int j = gt; j < taken; j += gn) {
    const int b = find(need, B, j);
    a.table[(size_t)b * a.max_pages + pages_for(ctx[b], a.page) + (j - need[b])] = a.free_pages[top - 1 - j];
  }
  // a thread takes four consecutive list entries: one search, then steps to the
  // next request; entries on one page share its look-up
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  for (int n0 = 4 * gt; n0 < a.n_slots; n0 += 4 * gn) {
    int slot[4], pos[4];
    int b = n0 < cu[B] ? find(cu, B, n0) : B;
    int first = -1, p = 0, off = P, page = 0, held = 0;  // the request the rest is about; next position, its place in its page
    bool served = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = n0 + k;
      slot[k] = pos[k] = -1;
      if (n >= a.n_slots || n >= cu[B]) continue;
      while (n >= cu[b + 1]) ++b;
      int pg = -1;  // the page to look up
      if (b != first) {
        first = b;
        held = pages_for(ctx[b], a.page);
        const bool fits = (long long)ctx[b] + (cu[b + 1] - cu[b]) <= row_tokens && cu[b + 1] <= a.n_slots;
        served = fits && (need[b + 1] == need[b] || need[b + 1] <= top);
        p = ctx[b] + (n - cu[b]);
        pg = a.page.quotient(p);
        off = p - pg * P;
      } else if (off == P) {
        pg = a.page.quotient(p);
        off = 0;
      }
      if (!served) continue;
      if (pg >= 0)
        page = pg < held ? a.table[(size_t)b * a.max_pages + pg] : a.free_pages[top - 1 - (need[b] + pg - held)];
      slot[k] = (uint32_t)page < (uint32_t)a.num_pages ? page * P + off : -1;  // a table entry may be no page
      pos[k] = p;
      ++p;
      ++off;
    }
    if (wide && n0 + 4 <= a.n_slots) {
      *reinterpret_cast<int4*>(a.slots + n0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + n0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int k = 0; k < 4 && n0 + k < a.n_slots; ++k) {
        a.slots[n0 + k] = slot[k];
        if (a.positions) a.positions[n0 + k] = pos[k];
      }
    }
  }
  for (int b = gt; b <= B; b += gn) {
    a.cu[b] = cu[b];
    if (b == B) break;
    const long long end = (long long)ctx[b] + (cu[b + 1] - cu[b]);
    const bool fits = end <= row_tokens && cu[b + 1] <= a.n_slots;
    a.lens[b] = fits && (need[b + 1] == need[b] || need[b + 1] <= top) ? (int)end : ctx[b];
  }
  if (gt == 0) *a.count_out = top - taken;
}

}  // namespace

static size_t plan_smem(int batch) { return sizeof(int) * (4 * (size_t)batch + 3); }

// The limit is the function's, not a call's: it is set once per device, to what the
// largest batch needs, and never lowered under another thread's launch
template <int TH>
static cudaError_t allow_smem() {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_page_plan<TH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kMaxPlanBatch));
    if (e == cudaSuccess && dev <= 63) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return e;
}

template <int TH>
static cudaError_t launch_sized(const PlanArgs& a, int ctas, cudaStream_t s) {
  const size_t smem = plan_smem(a.batch);
  if (smem > 48 * 1024) {
    cudaError_t e = allow_smem<TH>();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(TH);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_page_plan<TH>, a);
}

// The widest cluster this device can hold (16 CTAs of 1024 threads take that many SMs
// of one GPC), asked for once per device
static int plan_ctas() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return kPortable;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n) return n;
  int clusters = 0;
  n = kPortable;
  if (cudaFuncSetAttribute(k_page_plan<1024>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      allow_smem<1024>() == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    cfg.gridDim = dim3(kWidest);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = plan_smem(kMaxPlanBatch);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kWidest;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters, k_page_plan<1024>, &cfg) == cudaSuccess && clusters > 0) n = kWidest;
  }
  if (n == kPortable) cudaGetLastError();  // a refused question is not the caller's error
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  // us of one CTA of 256 threads, one of 1024, and a cluster: 5.1, 6.8 and 7.2 for 8
  // requests of one token; -, 6.8 and 7.1 for 64 of 60; -, 12.2 and 7.5 for 64 of 250.
  // The cluster of 16 against one of 8: 12.2 and 14.5 for 120,000 tokens, 21.8 and
  // 36 for 512,000.
  const long long work = (long long)a.n_slots + a.batch;
  if (work > 4096) return launch_sized<1024>(a, plan_ctas(), s);
  return work > 1024 ? launch_sized<1024>(a, 1, s) : launch_sized<256>(a, 1, s);
}

}  // namespace kvq
