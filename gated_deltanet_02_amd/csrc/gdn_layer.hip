// gfx950 (CDNA4) kernels around a recurrent layer's projections: the short
// causal convolution and the residual root-mean-square norm.  Both move each
// byte once and are bound by HBM (large calls) or by the launch and one trip
// to memory (small ones).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {

// ---------------------------------------------------------------------------
// The short convolution: y[t, c] = bias[c] + sum_j w[c][j] e[t + j, c] (e: a
// sequence's W - 1 history rows, then its rows), optionally silu.
//
// A thread takes 16 bytes' worth of adjacent channels (one element where
// vector accesses do not fit) and walks a tile of 32 tokens, the last W - 1
// rows in registers and the next four tokens' rows on their way, so a row is
// read once, but for the W - 1 rows before a tile, which its neighbour on the
// same XCD has in L2.  The taps lie channel by channel, 128 bytes apart for
// neighbouring lanes: read as they lie they would take as long as a tile's
// rows, so the workgroup reads them once in order and turns them in LDS.
//
// Measured (bf16, W = 4): 137k tokens x 6144 channels 637 us, 5.3 TB/s (a
// large copy reaches 4.8; 984 us in tiles of 64 with the taps read as they lie
// and no rows on their way); 256 steps of 6144 channels 8.7 us, the launch and
// the trips for the table, the rows and the taps.
//
// The tiles cut the tokens regardless of sequences and leave out each
// sequence's first W - 1 tokens: those, and the new history, belong to a
// second kind of work item, one per sequence, the only one that reads
// state_in and writes state_out, which may therefore be one array.

constexpr int kConvThreads = 256;
constexpr int kConvTile = 32;     // tokens per tile, fewer where tiles are few
constexpr int kConvGroup = 4;     // tokens asked for at once

template <typename TI, bool VEC>
struct ConvVec {
  static constexpr int n = VEC ? 16 / (int)sizeof(TI) : 1;
};

template <typename TI, bool VEC, int E>
__device__ __forceinline__ void conv_store(TI* p, const float (&v)[E]) {
  if constexpr (VEC) {
    uint4 r;
    TI* e = (TI*)&r;
#pragma unroll
    for (int i = 0; i < E; ++i) e[i] = from_float<TI>(v[i]);
    st16(p, r);
  } else {
    *p = from_float<TI>(v[0]);
  }
}

// Entry i of cu_seqlens, clamped into [0, t_total].
__device__ __forceinline__ int conv_cu(const ShortConvParams& p, int i) {
  const int64_t e = p.cu_i64 ? ((const int64_t*)p.cu)[i] : ((const int32_t*)p.cu)[i];
  return (int)min(max(e, (int64_t)0), (int64_t)p.t_total);
}

// The last of the sequences lo .. hi that starts at or before token t (lo if
// none does).
__device__ __forceinline__ int conv_find(const ShortConvParams& p, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = lo + ((hi - lo + 1) >> 1);  // (lo + hi can pass 2^31)
    if (conv_cu(p, mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// What a thread loads of a row, and its values.
template <typename TI, bool VEC>
struct ConvRaw {
  typename std::conditional<VEC, uint4, TI>::type v;
  __device__ __forceinline__ void load(const TI* p) { v = *(const decltype(v)*)p; }
  template <int E>
  __device__ __forceinline__ void get(float (&f)[E]) const {
    if constexpr (VEC) {
      const TI* e = (const TI*)&v;
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = to_float(e[i]);
    } else {
      f[0] = to_float(v);
    }
  }
};

// A workgroup takes `cols` threads' channels (a power of two) of 256 / cols
// work items; blocks_c workgroups cover the channels.
template <typename TI, int W, bool VEC>
__global__ __launch_bounds__(kConvThreads) void short_conv_kernel(ShortConvParams p, int cols, int blocks_c, int tile,
                                                                 int tiles_per_seq, int n_tiles) {
  constexpr int E = ConvVec<TI, VEC>::n;
  __shared__ __attribute__((aligned(16))) float s_w[W + 1][kConvThreads * E];
  // workgroups k, k + 8, ... run on one XCD: it takes an eighth of the work
  // in order, so that neighbouring tiles share an L2
  const unsigned per = (gridDim.x + 7) / 8, id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  const int cb = id % blocks_c, tx = threadIdx.x % cols;
  const int64_t item64 = p.first_item + (int64_t)(id / blocks_c) * (kConvThreads / cols) + threadIdx.x / cols;
  const int first = cb * cols * E;  // the workgroup's first channel
  const int c0 = first + tx * E;
  const bool live = item64 < p.end_item && c0 < p.d;
  const TI* x = (const TI*)p.x + c0;
  TI* out = (TI*)p.out + c0;
  // What a sequence's own item reads, asked for before the taps are turned:
  // the history, the first rows, the last rows.
  const int own = live && item64 >= n_tiles ? (int)(item64 - n_tiles) : -1;  // its sequence, or < 0: a tile
  int own_start = 0, own_len = 0;
  ConvRaw<TI, VEC> hist[W], head[W], tail[W];
  const TI* hin = nullptr;
  if (own >= 0) {
    if (p.cu) {
      own_start = conv_cu(p, own);
      own_len = max(conv_cu(p, own + 1) - own_start, 0);
    } else {
      own_start = own * p.seq_len;
      own_len = p.seq_len;
    }
    if (p.state_in) hin = (const TI*)p.state_in + (int64_t)own * (W - 1) * p.d + c0;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) {
      if (hin) hist[j].load(hin + (int64_t)j * p.d);
      if (j < own_len) head[j].load(x + (int64_t)(own_start + j) * p.x_st);
      if (own_len + j >= W - 1) tail[j].load(x + (int64_t)(own_start + own_len + j - (W - 1)) * p.x_st);
    }
  }
  {
    const int n = min(cols * E, p.d - first);
    float t[E][W + 1];
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int i = min((int)threadIdx.x + k * kConvThreads, n - 1);
#pragma unroll
      for (int j = 0; j < W; ++j) t[k][j] = p.w[(int64_t)(first + i) * W + j];
      t[k][W] = p.bias ? p.bias[first + i] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const int i = (int)threadIdx.x + k * kConvThreads;
#pragma unroll
      for (int j = 0; j <= W; ++j)
        if (i < n) s_w[j][i] = t[k][j];
    }
  }
  __syncthreads();
  if (!live) return;

  float w[W][E], bias[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    bias[e] = s_w[W][tx * E + e];
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][e] = s_w[j][tx * E + e];
  }
  // rows[j]: the raw row W - 1 - j tokens before the current one
  float rows[W][E];
  auto emit = [&](int64_t t, const float (*r)[E]) {
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float a = bias[e];
#pragma unroll
      for (int j = 0; j < W; ++j) a += w[j][e] * r[j][e];
      y[e] = p.silu ? silu_f32(a) : a;
    }
    conv_store<TI, VEC>(out + t * p.o_st, y);
  };
  auto shift = [&]() {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) rows[j][e] = rows[j + 1][e];
  };

  if (own < 0) {
    const int item = (int)item64;
    // tokens [t0, t1), the current sequence's start and end
    int t0, t1, start, end, seq = 0, last = 0;
    if (p.cu) {
      t0 = item * tile;
      t1 = min(t0 + tile, conv_cu(p, p.n_seq));
      last = p.n_seq - 1;
      seq = conv_find(p, 0, last, t0);
      start = conv_cu(p, seq);
      end = conv_cu(p, seq + 1);
    } else {
      seq = last = item / tiles_per_seq;
      start = seq * p.seq_len;
      end = start + p.seq_len;
      t0 = start + (item - seq * tiles_per_seq) * tile;
      t1 = min(t0 + tile, end);
    }
    if (t0 >= t1) return;
    ConvRaw<TI, VEC> before[W], next[kConvGroup];
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) before[j].load(x + (int64_t)max(t0 - (W - 1) + j, 0) * p.x_st);
    auto ask = [&](int t) {
#pragma unroll
      for (int i = 0; i < kConvGroup; ++i) next[i].load(x + (int64_t)min(t + i, t1 - 1) * p.x_st);
    };
    ask(t0);
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) before[j].get(rows[j]);
    for (int t = t0; t < t1; t += kConvGroup) {
      ConvRaw<TI, VEC> now[kConvGroup];
#pragma unroll
      for (int i = 0; i < kConvGroup; ++i) now[i] = next[i];
      ask(t + kConvGroup);
      if (t + kConvGroup <= min(t1, end) && t - start >= W - 1) {
        // a whole group inside a sequence: no rows change places in between
        float e[W - 1 + kConvGroup][E];
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
          for (int k = 0; k < E; ++k) e[j][k] = rows[j][k];
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i) now[i].get(e[W - 1 + i]);
#pragma unroll
        for (int i = 0; i < kConvGroup; ++i) emit(t + i, e + i);
#pragma unroll
        for (int j = 0; j + 1 < W; ++j)
#pragma unroll
          for (int k = 0; k < E; ++k) rows[j][k] = e[kConvGroup + j][k];
        continue;
      }
#pragma unroll
      for (int i = 0; i < kConvGroup; ++i) {
        if (t + i >= t1) break;
        if (t + i >= end && seq < last) {
          start = conv_cu(p, ++seq);
          end = conv_cu(p, seq + 1);
          if (t + i >= end) {  // the one behind a run of empty ones
            seq = conv_find(p, seq, last, t + i);
            start = conv_cu(p, seq);
            end = conv_cu(p, seq + 1);
          }
        }
        now[i].get(rows[W - 1]);
        if (t + i - start >= W - 1) emit(t + i, rows);
        shift();
      }
    }
    return;
  }

  // A sequence's first W - 1 tokens and its new history.
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) {
#pragma unroll
    for (int e = 0; e < E; ++e) rows[j][e] = 0.f;
    if (hin) hist[j].get(rows[j]);
  }
  float old[W][E];
#pragma unroll
  for (int j = 0; j + 1 < W; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) old[j][e] = rows[j][e];
#pragma unroll
  for (int i = 0; i + 1 < W; ++i) {
    if (i < own_len) {
      head[i].get(rows[W - 1]);
      emit(own_start + i, rows);
      shift();
    }
  }
  if (!p.state_out) return;
  TI* hout = (TI*)p.state_out + (int64_t)own * (W - 1) * p.d + c0;
#pragma unroll
  for (int j = 0; j + 1 < W; ++j) {
    // row len + j of the history followed by the sequence
    float v[E];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k)
      if (k == own_len + j)
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = old[k][e];
    if (own_len + j >= W - 1) tail[j].get(v);
    conv_store<TI, VEC>(hout + (int64_t)j * p.d, v);
  }
}

template <typename TI, bool VEC>
static hipError_t launch_short_conv_t(const ShortConvParams& all, hipStream_t s) {
  constexpr int E = ConvVec<TI, VEC>::n;
  const int64_t nvec = (all.d + E - 1) / E;
  int cols = 1;
  while (cols < nvec && cols < kConvThreads) cols *= 2;
  const int64_t blocks_c = (nvec + cols - 1) / cols;
  // shorter tiles where the long ones would leave compute units with less
  // than one workgroup each per SIMD (1237 rows of 1001 channels: 9.2 us in
  // tiles of 32, 6.1 us in tiles of 8)
  int tile = kConvTile;
  while (tile > 2 * kConvGroup && (int64_t)all.t_total / tile * nvec < 1024 * kConvThreads) tile /= 2;
  // sequences of fewer than W tokens have no tokens for the tiles
  const int64_t per_seq = all.cu ? 0 : all.seq_len < all.width ? 0 : (all.seq_len + tile - 1) / tile;
  const int64_t tiles = all.cu ? ((int64_t)all.t_total + tile - 1) / tile : per_seq * all.n_seq;
  const int64_t items = tiles + all.n_seq, per_block = kConvThreads / cols;
  // over as many launches as the items take (in any order: an item reads and
  // writes no other's history)
  const int64_t most = (kLaunchThreads / kConvThreads - 7) / blocks_c * per_block;
  for (int64_t first = 0; first < items; first += most) {
    ShortConvParams p = all;
    p.first_item = first;
    const int64_t n = items - first < most ? items - first : most;
    p.end_item = first + n;
    const int64_t blocks = ((n + per_block - 1) / per_block * blocks_c + 7) / 8 * 8;
    switch (p.width) {
#define GDN_CONV(W)                                                                                        \
      case W:                                                                                              \
        hipLaunchKernelGGL((short_conv_kernel<TI, W, VEC>), dim3((unsigned)blocks), dim3(kConvThreads), 0, s, p, \
                           cols, (int)blocks_c, tile, (int)per_seq, (int)tiles);                           \
        break;
      GDN_CONV(1) GDN_CONV(2) GDN_CONV(3) GDN_CONV(4)
#undef GDN_CONV
      default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_short_conv(bool bf16, bool vec, const ShortConvParams& p, hipStream_t s) {
  if (bf16) return vec ? launch_short_conv_t<gdn::bf16, true>(p, s) : launch_short_conv_t<gdn::bf16, false>(p, s);
  return vec ? launch_short_conv_t<float, true>(p, s) : launch_short_conv_t<float, false>(p, s);
}

// ---------------------------------------------------------------------------
// The residual norm: r = x + residual, y = r / sqrt(mean r^2 + eps) * w, with
// y in the input's type, in e4m3 with a scale per row or per 128 columns, or
// both.
//
// TPR threads hold a row in registers, each NV vectors of eight adjacent
// columns, so the row is read once and the two reductions (the sum of
// squares; the largest |y|, of a row, or of the 16 lanes that hold a group)
// run on registers.  Rows of up to 1024 columns take one wave each, longer
// ones a workgroup.  Measured: 4096 rows of 5120 columns in bf16 with residual
// and both outputs 44 us, 4.3 TB/s; 131071 rows of 6144 with 8-bit output
// alone 932 us, 6.1 TB/s; eight rows 3.9 us, the launch, one trip and the
// reductions.

constexpr int kNormVec = 8;
constexpr float kE4m3Max = 448.f;
constexpr float kNormLeast = 0x1p-100f;   // mean squares from here on lose no digits to underflow
constexpr float kScaleFloor = 0x1p-100f;  // keeps a scale and its reciprocal finite

// The larger of two non-negative floats; a NaN (its bits are the larger
// integer) wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}

// 16-byte accesses, past the caches where FAR.
typedef unsigned norm_u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned norm_u32x4 __attribute__((ext_vector_type(4)));

template <typename V, bool FAR>
__device__ __forceinline__ V norm_ld(const void* p) {
  return FAR ? __builtin_nontemporal_load((const V*)p) : *(const V*)p;
}

template <bool FAR, typename V>
__device__ __forceinline__ void norm_st(void* p, V v) {
  if constexpr (FAR) __builtin_nontemporal_store(v, (V*)p);
  else *(V*)p = v;
}

// Eight columns from c0 on, those at or after d as zeros.
template <typename TI, bool VEC, bool FAR = false>
__device__ __forceinline__ void norm_load(float (&v)[kNormVec], const TI* row, int c0, int d) {
  if constexpr (VEC) {
    if constexpr (sizeof(TI) == 2) {
      const norm_u32x4 r = norm_ld<norm_u32x4, FAR>(row + c0);
      const TI* e = (const TI*)&r;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
    } else {
      const f32x4 a = norm_ld<f32x4, FAR>(row + c0), b = norm_ld<f32x4, FAR>(row + c0 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < d ? to_float(row[c0 + i]) : 0.f;
  }
}

template <typename TI, bool VEC, bool FAR>
__device__ __forceinline__ void norm_store(TI* row, const float (&v)[kNormVec], int c0, int d) {
  if constexpr (VEC) {
    if constexpr (sizeof(TI) == 2) {
      norm_u32x4 r;
      TI* e = (TI*)&r;
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = from_float<TI>(v[i]);
      norm_st<FAR>(row + c0, r);
    } else {
      f32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = v[i];
        b[i] = v[4 + i];
      }
      norm_st<FAR>(row + c0, a);
      norm_st<FAR>(row + c0 + 4, b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < d) row[c0 + i] = from_float<TI>(v[i]);
  }
}

// Eight columns over their scale as e4m3 (the hardware conversion rounds to
// nearest even; |v / scale| is at most 448 up to fp32 rounding, and everything
// below 464 rounds into the range).  The fp32 quotient is the rounded one:
// v (1 / scale) corrected once by its remainder, without which codes next to
// a tie would flip.  (Under an infinite scale nothing is left but v * 0.)
template <bool VEC, bool FAR>
__device__ __forceinline__ void norm_store_q(uint8_t* row, const float (&v)[kNormVec], float scale, int c0,
                                             int d) {
  const float inv = 1.f / scale, by = scale < __builtin_inff() ? scale : 0.f;
  float u[kNormVec];
#pragma unroll
  for (int i = 0; i < kNormVec; ++i) {
    const float q = v[i] * inv;
    u[i] = __builtin_fmaf(-__builtin_fmaf(q, by, -v[i]), inv, q);  // (keeps the sign of a zero)
  }
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(u[0], u[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(u[2], u[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(u[4], u[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(u[6], u[7], b, true);
  if constexpr (VEC) {
    norm_st<FAR>(row + c0, (norm_u32x2){(unsigned)a, (unsigned)b});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < d) row[c0 + i] = (uint8_t)((i < 4 ? a : b) >> (8 * (i & 3)));
  }
}

// A reduction over the TPR threads of a row (one wave, or the workgroup).
template <int TPR, typename F>
__device__ __forceinline__ float row_reduce(float v, float* lds, F f) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = f(v, __shfl_xor(v, off));
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = f(v, lds[i]);
  }
  return v;
}

template <typename TI, int TPR, int NV, bool VEC, bool FAR>
__global__ __launch_bounds__(TPR > 64 ? TPR : 256) void add_rms_norm_kernel(NormParams p) {
  constexpr int RPB = TPR > 64 ? 1 : 4;  // rows per workgroup
  __shared__ float s_sum[16], s_max[16], s_again[16];
  const int sub = TPR > 64 ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * RPB + (TPR > 64 ? 0 : threadIdx.x >> 6);
  if (row >= p.rows) return;
  const TI* x = (const TI*)p.x + row * p.x_st;
  const TI* res = p.res ? (const TI*)p.res + row * p.r_st : nullptr;
  float v[NV][kNormVec];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = (sub + i * TPR) * kNormVec;
#pragma unroll
    for (int e = 0; e < kNormVec; ++e) v[i][e] = 0.f;
    if (c0 < p.d) {
      norm_load<TI, VEC, FAR>(v[i], x, c0, p.d);
      if (res) {
        float r[kNormVec];
        norm_load<TI, VEC, FAR>(r, res, c0, p.d);
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) v[i][e] += r[e];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = (sub + i * TPR) * kNormVec;
    if (p.res_out && c0 < p.d) norm_store<TI, VEC, FAR>((TI*)p.res_out + row * p.ro_st, v[i], c0, p.d);
#pragma unroll
    for (int e = 0; e < kNormVec; ++e) ss += v[i][e] * v[i][e];
  }
  ss = row_reduce<TPR>(ss, s_sum, [](float a, float b) { return a + b; });
  float eps = p.eps, mean = ss / (float)p.d;
  if (!(mean + eps >= kNormLeast && mean < __builtin_inff())) {
    // squares past fp32's range (or NaN, or real infinities, which give the
    // same again): once more, of the row times a power of two
    const float by = mean < 1.f ? 0x1p100f : 0x1p-76f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < kNormVec; ++e) {
        v[i][e] *= by;
        ss += v[i][e] * v[i][e];
      }
    mean = row_reduce<TPR>(ss, s_again, [](float a, float b) { return a + b; }) / (float)p.d;
    eps = eps * by * by;
  }
  const float rn = 1.f / sqrtf(mean + eps);
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = (sub + i * TPR) * kNormVec;
    const bool live = c0 < p.d;
    float top = 0.f;
    if (live) {
      float w[kNormVec];
      if (p.w) {
        norm_load<float, VEC>(w, p.w, c0, p.d);
      } else {
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) w[e] = 1.f;
      }
#pragma unroll
      for (int e = 0; e < kNormVec; ++e) {
        v[i][e] = v[i][e] * rn * w[e];
        if (VEC || c0 + e < p.d) top = max_nan(top, fabsf(v[i][e]));
      }
      if (p.out) norm_store<TI, VEC, FAR>((TI*)p.out + row * p.o_st, v[i], c0, p.d);
    }
    if (p.out_q && p.groups) {
      // a group's 128 columns are 16 adjacent lanes, all of them here (those
      // past the row's end with a maximum of zero)
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) top = max_nan(top, __shfl_xor(top, off));
      const float scale = max_nan(top, kScaleFloor) / kE4m3Max;
      if (live) {
        norm_store_q<VEC, FAR>(p.out_q + row * p.q_st, v[i], scale, c0, p.d);
        if ((sub & 15) == 0) p.scales[row * p.groups + c0 / 128] = scale;
      }
    }
    big = max_nan(big, top);
  }
  if (p.out_q && !p.groups) {
    big = row_reduce<TPR>(big, s_max, [](float a, float b) { return max_nan(a, b); });
    const float scale = max_nan(big, kScaleFloor) / kE4m3Max;
    if (sub == 0) p.scales[row] = scale;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (sub + i * TPR) * kNormVec;
      if (c0 < p.d) norm_store_q<VEC, FAR>(p.out_q + row * p.q_st, v[i], scale, c0, p.d);
    }
  }
}

template <typename TI, bool VEC, bool FAR>
static hipError_t launch_add_rms_norm_t(const NormParams& p, hipStream_t s) {
  const int vecs = (p.d + kNormVec - 1) / kNormVec;
  const bool wave = vecs <= 128;
  const int64_t blocks = wave ? (p.rows + 3) / 4 : p.rows;
#define GDN_NORM(TPR, NV)                                                                             \
  do {                                                                                                \
    hipLaunchKernelGGL((add_rms_norm_kernel<TI, TPR, NV, VEC, FAR>), dim3((unsigned)blocks),                \
                       dim3(TPR > 64 ? TPR : 256), 0, s, p);                                          \
    return hipGetLastError();                                                                         \
  } while (0)
  if (vecs <= 64) GDN_NORM(64, 1);
  if (vecs <= 128) GDN_NORM(64, 2);
  if (vecs <= 256) GDN_NORM(256, 1);
  if (vecs <= 512) GDN_NORM(256, 2);
  if (vecs <= 768) GDN_NORM(256, 3);
  if (vecs <= 1024) GDN_NORM(256, 4);
  if (vecs <= 2048) GDN_NORM(1024, 2);
  if (vecs <= 4096) GDN_NORM(1024, 4);
  if (vecs <= 8192) GDN_NORM(1024, 8);
#undef GDN_NORM
  return hipErrorInvalidValue;
}

template <typename TI>
static hipError_t launch_add_rms_norm_v(bool vec, bool far, const NormParams& p, hipStream_t s) {
  if (!vec) return launch_add_rms_norm_t<TI, false, false>(p, s);
  return far ? launch_add_rms_norm_t<TI, true, true>(p, s) : launch_add_rms_norm_t<TI, true, false>(p, s);
}

hipError_t launch_add_rms_norm(bool bf16, bool vec, const NormParams& all, hipStream_t s) {
  const int64_t size = bf16 ? 2 : 4;
  // What the memory-side cache (256 MiB) cannot hold between this operator
  // and its neighbours goes past the caches: 131071 rows of 6144 (5.7 GB)
  // 994 -> 932 us, 16384 of 5120 with their neighbours 226 -> 209; below, the
  // neighbours lose what this operator gains (4096 rows 34 -> 30 us alone,
  // 59 -> 61 with them; 256 rows 6.4 -> 7.2).
  const int64_t bytes = all.rows * all.d * (size * (1 + !!all.res + !!all.res_out + !!all.out) + !!all.out_q);
  const bool far = bytes > (int64_t)256 << 20;
  constexpr int64_t most = (int64_t)1 << 21;  // rows of a launch, a row taking at most 1024 threads
  for (int64_t row = 0; row < all.rows; row += most) {
    NormParams p = all;
    auto at = [&](auto* a, int64_t bytes) { return a ? (decltype(a))((uintptr_t)a + row * bytes) : a; };
    p.rows = all.rows - row < most ? all.rows - row : most;
    p.x = at(all.x, all.x_st * size);
    p.res = at(all.res, all.r_st * size);
    p.res_out = at(all.res_out, all.ro_st * size);
    p.out = at(all.out, all.o_st * size);
    p.out_q = at(all.out_q, all.q_st);
    p.scales = at(all.scales, (all.groups ? all.groups : 1) * 4);
    const hipError_t e = bf16 ? launch_add_rms_norm_v<gdn::bf16>(vec, far, p, s) : launch_add_rms_norm_v<float>(vec, far, p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gdn
