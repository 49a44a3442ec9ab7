// The bookkeeping of a paged key-value cache on gfx950: block tables and slot
// maps from request lengths, the release of finished requests' pages, and the
// store of new rows.
//
// Plan.  Request i holds ceil(ctx_i / S) pages of S tokens and needs
// ceil((ctx_i + new_i) / S); with upto_i the running sum of the differences,
// it takes the pages from n_free - upto_i + diff_i - 1 downwards off the stack
// of free ones, and is served if upto_i <= n_free (or it needs none).  A fresh
// page's id follows from the sum alone, so every token finds its slot by
// itself: no pass waits for another.  What bounds it is latency: one launch
// for decode batches, whose workgroup keeps the sums in LDS.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn.h"
#include "gdn_device.h"

namespace gdn {

namespace {

constexpr int kLaunchMax = 1 << 23;  // workgroups of a launch (at most 256 threads each: 2^31)
constexpr int kPlanThreads = 512;
constexpr int kReleaseThreads = 1024;

__device__ __forceinline__ int quotient(const Divide& d, int n) {
  return (int)((__umulhi(d.mul, (uint32_t)n) + (uint32_t)n) >> d.shift);
}
__device__ __forceinline__ int quotient_up(const Divide& d, int n) { return n > 0 ? quotient(d, n - 1) + 1 : 0; }

__device__ __forceinline__ int cu_at(const void* cu, int i64, int64_t i, int t) {
  const int64_t v = i64 ? ((const int64_t*)cu)[i] : (int64_t)((const int32_t*)cu)[i];
  return (int)min(max(v, (int64_t)0), (int64_t)t);
}

// A request: its tokens before and its new ones, the pages it holds, and those
// it takes (0 where its table has no room: `fits` false).
struct Request {
  int ctx, start, fresh, have, extra;
  bool fits;
};

__device__ __forceinline__ Request request(const PlanParams& p, int i) {
  Request r;
  r.ctx = max(p.ctx[i], 0);
  if (p.cu) {
    r.start = cu_at(p.cu, p.cu_i64, i, p.t);
    r.fresh = max(cu_at(p.cu, p.cu_i64, i + 1, p.t) - r.start, 0);
  } else {
    r.start = i;
    r.fresh = 1;
  }
  r.have = quotient_up(p.page, r.ctx);
  const int64_t end = (int64_t)r.ctx + r.fresh;
  const int need = quotient_up(p.page, (int)min(end, (int64_t)INT32_MAX));
  r.fits = need <= p.width && end <= INT32_MAX;
  r.extra = r.fits ? need - r.have : 0;
  return r;
}

// Exclusive sums over the workgroup's threads, and the whole sum.
template <int THREADS>
__device__ __forceinline__ int64_t sums_before(int64_t v, int64_t* waves, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t upto = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  *total = all;
  return before + upto - v;
}

// Writes the lengths and what is left free (one workgroup): thread l's
// requests are [l c, (l + 1) c), with the sum before them.
__device__ __forceinline__ void plan_finish(const PlanParams& p, int c, int64_t before, int64_t n_free) {
  __shared__ int taken;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  int64_t upto = before;
  int mine = 0;
  const int64_t end = min((int64_t)(threadIdx.x + 1) * c, (int64_t)p.n);
  for (int64_t i = (int64_t)threadIdx.x * c; i < end; ++i) {
    const Request r = request(p, (int)i);
    upto += r.extra;
    const bool served = r.fits && (r.extra == 0 || upto <= n_free);
    p.lens[i] = served ? r.ctx + r.fresh : r.ctx;
    if (served && r.extra > 0) mine = (int)upto;
  }
  atomicMax(&taken, mine);
  __syncthreads();
  if (threadIdx.x == 0) p.n_free_out[0] = (int)n_free - taken;
}

// FINISH: the first workgroup also writes the lengths, once all its reads are
// done; where they are the ones read, it is the only one.
template <bool FINISH>
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(PlanParams p, int tokens) {
  __shared__ int64_t before[kPlanThreads], waves[kPlanThreads / 64];
  const int c = (int)(((int64_t)p.n + kPlanThreads - 1) / kPlanThreads);
  const int64_t n_free = min(max(p.n_free[0], 0), p.free_max);
  int64_t sum = 0, total;
  const int64_t end = min((int64_t)(threadIdx.x + 1) * c, (int64_t)p.n);
  for (int64_t i = (int64_t)threadIdx.x * c; i < end; ++i) sum += request(p, (int)i).extra;
  const int64_t mine = sums_before<kPlanThreads>(sum, waves, &total);
  before[threadIdx.x] = mine;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * tokens;
  const int64_t last = min(first + tokens, (int64_t)p.t);
  for (int64_t t = first + threadIdx.x; t < last; t += kPlanThreads) {
    int64_t i = t;
    if (p.cu) {
      // the last request that starts at or before t
      int64_t lo = 0, hi = p.n - 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu_at(p.cu, p.cu_i64, mid, p.t) <= t) lo = mid;
        else hi = mid - 1;
      }
      i = lo;
    }
    const Request r = request(p, (int)i);
    int64_t slot = -1;
    if (t >= r.start && t - r.start < r.fresh && r.fits) {
      const int at = r.ctx + (int)(t - r.start);
      const int col = quotient(p.page, at), in = at - col * (int)p.page.d;
      int64_t page = -1;
      if (col < r.have) {
        // (held pages are there whether the request is served or not)
        page = p.table[i * p.table_st + col];
      }
      if (r.extra > 0) {
        int64_t upto = before[(int)i / c];
        for (int j = (int)i / c * c; j < i; ++j) upto += request(p, j).extra;
        if (upto + r.extra > n_free) {
          page = -1;
        } else if (col >= r.have) {
          page = p.free[n_free - 1 - upto - (col - r.have)];
          if (in == 0) p.table[i * p.table_st + col] = (int32_t)page;
        }
      }
      if (page >= 0) slot = page * p.page.d + in;
    }
    p.slots[t] = slot;
  }
  if constexpr (FINISH) {
    if (blockIdx.x > 0) return;
    __syncthreads();
    plan_finish(p, c, mine, n_free);
  }
}

__global__ __launch_bounds__(kPlanThreads) void plan_finish_kernel(PlanParams p) {
  __shared__ int64_t waves[kPlanThreads / 64];
  const int c = (int)(((int64_t)p.n + kPlanThreads - 1) / kPlanThreads);
  const int64_t n_free = min(max(p.n_free[0], 0), p.free_max);
  int64_t sum = 0, total;
  const int64_t end = min((int64_t)(threadIdx.x + 1) * c, (int64_t)p.n);
  for (int64_t i = (int64_t)threadIdx.x * c; i < end; ++i) sum += request(p, (int)i).extra;
  const int64_t mine = sums_before<kPlanThreads>(sum, waves, &total);
  __syncthreads();
  plan_finish(p, c, mine, n_free);
}

// The finished requests' pages back on the stack, in the order of the
// requests; a round takes as many requests as there are threads, dealt out to
// the waves, eight pieces of 64 entries at a time.  Entries below 0 name no page
// and have no place on the stack: the pages are counted before any is written.
// Bound by one workgroup's instructions and waits: 256 requests of 125 pages 13.8
// us, 64 of 2048 18, 4096 of 13 126.
__global__ __launch_bounds__(kReleaseThreads) void release_kernel(ReleaseParams p) {
  constexpr int WAVES = kReleaseThreads / 64, BATCH = 8;
  static_assert(WAVES * 64 == kReleaseThreads, "a row a lane");
  __shared__ int64_t waves[WAVES], at_of[kReleaseThreads];
  __shared__ int entries_of[kReleaseThreads];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int mine = wave + WAVES * lane;  // the lane's among the wave's requests
  int64_t top = min(max(p.n_free[0], 0), p.free_max);
  for (int64_t i0 = 0; i0 < p.n; i0 += kReleaseThreads) {
    const int64_t i = i0 + threadIdx.x;
    int entries = 0;
    if (i < p.n && p.done[i]) {
      entries = min(quotient_up(p.page, max(p.lens[i], 0)), p.width);
      p.lens[i] = 0;
    }
    entries_of[threadIdx.x] = entries;
    __syncthreads();
    entries = entries_of[mine];
    const int over = entries % (64 * BATCH), whole = entries - over;
    const uint64_t some = __ballot(over > 0);
    int32_t* const rows = p.table + (i0 + wave) * p.table_st + lane;
    const int64_t step = WAVES * p.table_st;
    // what(the request's lane, entry, whether there is one, its address) for all
    // pieces of the wave's requests: whole batches of a request, then what is
    // over, of several requests a batch
    const auto each = [&](const auto& what) {
      int32_t e[BATCH];
      for (uint64_t left = __ballot(whole > 0); left; left &= left - 1) {
        const int k = __ffsll((unsigned long long)left) - 1, n = __builtin_amdgcn_readlane(whole, k);
        int32_t* from = rows + k * step;
        for (int j = 0; j < n; j += 64 * BATCH, from += 64 * BATCH) {
#pragma unroll
          for (int b = 0; b < BATCH; ++b) e[b] = from[64 * b];
#pragma unroll
          for (int b = 0; b < BATCH; ++b) what(k, e[b], true, from + 64 * b);
        }
      }
      int k = 64, n = 0;
      int32_t* from = nullptr;
      uint64_t left = some;
      const auto next = [&] {  // (k = 64: none)
        k = left ? __ffsll((unsigned long long)left) - 1 : 64;
        left &= left - 1;
        n = k < 64 ? __builtin_amdgcn_readlane(over, k & 63) : 0;
        from = rows + k * step + __builtin_amdgcn_readlane(whole, k & 63);
      };
      for (next(); k < 64;) {
        int at[BATCH];
        int32_t* place[BATCH];
        bool is[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
          at[b] = k;
          place[b] = from;
          is[b] = lane < n;
          e[b] = is[b] ? *from : -1;
          n -= 64;
          from += 64;
          if (n <= 0) next();
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) what(at[b], e[b], is[b], place[b]);
      }
    };
    int pages = 0;
    each([&](int k, int32_t e, bool, int32_t*) {
      const int held = __popcll(__ballot(e >= 0));
      pages += lane == k ? held : 0;
    });
    at_of[mine] = pages;
    __syncthreads();
    int64_t total;
    const int64_t before = sums_before<kReleaseThreads>(at_of[threadIdx.x], waves, &total);
    at_of[threadIdx.x] = top + before;
    __syncthreads();
    const int64_t first = at_of[mine];
    int done = 0;  // of the lane's pages
    each([&](int k, int32_t e, bool is, int32_t* place) {
      const uint64_t held = __ballot(e >= 0);
      const int64_t to = (((int64_t)__builtin_amdgcn_readlane((int)(first >> 32), k & 63) << 32) |
                          (uint32_t)__builtin_amdgcn_readlane((int)first, k & 63)) +
                         __builtin_amdgcn_readlane(done, k & 63) +
                         (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(held >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)held, 0));
      if (e >= 0 && to < p.free_max) p.free[to] = e;
      if (is) *place = -1;
      const int count = __popcll(held);
      done += lane == k ? count : 0;
    });
    __syncthreads();
    top += total;
  }
  if (threadIdx.x == 0) p.n_free[0] = (int32_t)min(top, (int64_t)p.free_max);
}

}  // namespace

hipError_t launch_cache_plan(const PlanParams& p, hipStream_t s) {
  // Workgroups each sum all requests.  One token a thread (64 prompts of 131072
  // tokens in all: 6.8 us of the kernel; four 12.7), four where the sums are long.
  const bool apart = p.lens != p.ctx && p.n_free_out != p.n_free;
  const int tokens = p.n > 16 * kPlanThreads || (!apart && p.t <= 4 * kPlanThreads) ? 4 * kPlanThreads : kPlanThreads;
  const int64_t groups = std::max<int64_t>(((int64_t)p.t + tokens - 1) / tokens, 1);
  if (groups == 1 || apart) {
    hipLaunchKernelGGL(plan_kernel<true>, dim3((unsigned)groups), dim3(kPlanThreads), 0, s, p, tokens);
    return hipGetLastError();
  }
  // lengths or a count that every workgroup reads are written in a launch of
  // their own
  hipLaunchKernelGGL(plan_kernel<false>, dim3((unsigned)groups), dim3(kPlanThreads), 0, s, p, tokens);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(plan_finish_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_cache_release(const ReleaseParams& p, hipStream_t s) {
  hipLaunchKernelGGL(release_kernel, dim3(1), dim3(kReleaseThreads), 0, s, p);
  return hipGetLastError();
}

namespace {

// A token's rows of k, then of v, a 16-byte granule a thread.  Bound by memory
// where a token fills its workgroup (137k tokens, 8 heads of 128: 183 us, 6.1
// TB/s), by the number of workgroups where it does not (1 head of 64: 54 us, 1.3).
__global__ __launch_bounds__(256) void store_kernel(StoreParams p, int64_t first) {
  const int per = p.kv << p.row_shift;  // granules of k of a token
  const int64_t t = first + blockIdx.x;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.n_slots) return;
  const int64_t page = slot <= INT32_MAX ? quotient(p.page, (int)slot) : slot / p.page.d, in = slot - page * p.page.d;
  const char* k = (const char*)p.k + t * p.k_st;
  const char* v = (const char*)p.v + t * p.v_st;
  char* kc = (char*)p.k_cache + page * p.kc_sp + in * p.kc_st;
  char* vc = (char*)p.v_cache + page * p.vc_sp + in * p.vc_st;
  for (int g = threadIdx.x; g < 2 * per; g += 256) {
    const bool second = g >= per;
    const int i = second ? g - per : g;
    const int h = i >> p.row_shift, o = (i & ((1 << p.row_shift) - 1)) * 16;
    const char* src = second ? v + h * p.v_sh + o : k + h * p.k_sh + o;
    char* dst = second ? vc + h * p.vc_sh + o : kc + h * p.kc_sh + o;
    st16(dst, ld16(src));
  }
}

}  // namespace

hipError_t launch_cache_store(const StoreParams& p, hipStream_t s) {
  for (int64_t first = 0; first < p.t; first += kLaunchMax) {
    const int64_t n = std::min<int64_t>(p.t - first, kLaunchMax);
    hipLaunchKernelGGL(store_kernel, dim3((unsigned)n), dim3(256), 0, s, p, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gdn
