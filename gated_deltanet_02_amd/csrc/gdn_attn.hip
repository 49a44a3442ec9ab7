// Attention of prompts and of single tokens over a paged key-value cache on
// gfx950: out = softmax(scale q.k) v over the keys that a query sees, those
// at or before its place and, with a window, inside it or among the first
// `sinks`.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn.h"
#include "gdn_tiles.h"

namespace gdn {

namespace {

__device__ __forceinline__ int attn_quotient(const Divide& d, int n) {
  return (int)((__umulhi(d.mul, (uint32_t)n) + (uint32_t)n) >> d.shift);
}

__device__ __forceinline__ int attn_cu(const AttnParams& p, int64_t i) {
  const int64_t v = p.cu_i64 ? ((const int64_t*)p.cu)[i] : (int64_t)((const int32_t*)p.cu)[i];
  return (int)min(max(v, (int64_t)0), (int64_t)p.t_total);
}

// One wave a row and head: lanes share a row's d, keys one after the other.
template <typename TI, int D, bool STEP>
__global__ __launch_bounds__(256) void attn_plain(AttnParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = item / p.heads;
  const int h = (int)(item - t * p.heads);
  if (t >= p.t_total) return;
  int seq, place, start = 0;
  if (STEP) {
    seq = (int)t;
    place = min(max(p.lens[seq], 0), p.max_len) - 1;
  } else {
    int end;
    if (p.cu) {
      int lo = 0, hi = p.n_seq - 1;
      while (lo < hi) {
        const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
        if (attn_cu(p, mid) <= t) lo = mid;
        else hi = mid - 1;
      }
      seq = lo;
      start = attn_cu(p, seq);
      end = attn_cu(p, seq + 1);
    } else {
      seq = (int)(t / p.seq_len);
      start = seq * p.seq_len;
      end = start + p.seq_len;
    }
    if (t < start || t >= end) return;
    place = (int)t - start;
    if (p.table) place += min(max(p.lens[seq], 0), p.max_len) - (end - start);
  }
  const char* q = (const char*)p.q + t * p.q_st + h * p.q_sh;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = to_float(((const TI*)q)[lane + 64 * e]);
    o[e] = 0.f;
  }
  const int kh = h / p.group;
  for (int j = 0; j <= place; ++j) {
    if (p.window > 0 && place - j >= p.window && j >= p.sinks) {
      j = place - p.window;
      continue;
    }
    const char *kr, *vr;
    if (p.table) {
      const int c = attn_quotient(p.page, j), in = j - c * (int)p.page.d;
      const int page = p.table[seq * p.table_st + c];
      if (page < 0 || page >= p.pages) continue;
      kr = (const char*)p.k + page * p.k_sp + in * p.k_st;
      vr = (const char*)p.v + page * p.v_sp + in * p.v_st;
    } else {
      kr = (const char*)p.k + (int64_t)(start + j) * p.k_st;
      vr = (const char*)p.v + (int64_t)(start + j) * p.v_st;
    }
    kr += kh * p.k_sh;
    vr += kh * p.v_sh;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qv[e] * to_float(((const TI*)kr)[lane + 64 * e]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    s *= p.scale;
    const float top = fmaxf(m, s), old = __builtin_amdgcn_exp2f(m - top), w = __builtin_amdgcn_exp2f(s - top);
    m = top;
    l = l * old + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * old + w * to_float(((const TI*)vr)[lane + 64 * e]);
  }
  TI* out = (TI*)((char*)p.out + t * p.o_st + h * p.o_sh);
#pragma unroll
  for (int e = 0; e < E; ++e) out[lane + 64 * e] = from_float<TI>(l > 0.f ? o[e] / l : o[e]);
}

template <bool STEP>
hipError_t launch_plain(bool bf16_in, int d, const AttnParams& p, hipStream_t s) {
  const dim3 grid((unsigned)(((int64_t)p.t_total * p.heads + 3) / 4)), threads(256);
  const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, threads, 0, s, p); };
  if (d == 64) bf16_in ? go(attn_plain<bf16, 64, STEP>) : go(attn_plain<float, 64, STEP>);
  else if (d == 128) bf16_in ? go(attn_plain<bf16, 128, STEP>) : go(attn_plain<float, 128, STEP>);
  else bf16_in ? go(attn_plain<bf16, 256, STEP>) : go(attn_plain<float, 256, STEP>);
  return hipGetLastError();
}

}  // namespace

int attn_tile_rows(bool, int) { return 128; }
hipError_t launch_attn_prefill(bool bf16_in, int d, const AttnParams& p, hipStream_t s) {
  return launch_plain<false>(bf16_in, d, p, s);
}

int attn_decode_waves(bool, int) { return 1024; }
hipError_t launch_attn_decode(bool bf16_in, int d, const AttnParams& p, hipStream_t s) {
  return launch_plain<true>(bf16_in, d, p, s);
}

}  // namespace gdn
