// gfx950 (CDNA4) kernels of the selective state space scan:
//   S_t = e^(g_t) S_{t-1} + d_t b_t x_t^T  (N x P),  y_t = S_t^T c_t + D x_t,
//   d_t = softplus(dt_t + bias),  g_t = -e^(a_log) d_t,
// per packed sequence and head.
//
// Summed over a block of C tokens with cum_i = g_0 + ... + g_i (inside the
// block) and S the state before it:
//   y_i = e^(cum_i) S^T c_i + sum_{j <= i} M_ij x_j,
//   M_ij = (c_i . b_j) e^(cum_i - cum_j) d_j  (+ D on the diagonal),
//   S  <- e^(cum_last) S + sum_t b_t (w_t x_t)^T,  w_t = e^(cum_last - cum_t) d_t,
// four matrix products per block, on the matrix cores.  Every exponent is a
// difference taken inside a block and <= 0.
//
// Precision.  In each product one operand is an input as stored (exact); the
// other is fp32 and is fed as the sum of bf16 terms: two for the outputs (M
// and S; 2^-17 of a product, below the output's own rounding), three for the
// state (w_t x_t; 2^-25, so the fp32 state keeps fp32 accuracy).  The extra
// matrix instructions stay under the time the block's bytes take.  fp32
// inputs use fp32 matrix instructions throughout.
//
// A workgroup scans one segment of one head, the state in the accumulators
// of its waves (each wave holds all N rows of its CW columns).  The fragment
// layout along the contraction index is the accumulators' own (k-tile order,
// gdn_device.h), so the state and x feed the products without leaving their
// lanes; b and c are stored in LDS with that order inside each row, x in its
// own order and read transposed.
//
// A sequence cut into segments takes three launches: the segments' end
// states from zero (the same kernel without c and y), their joining in
// order, and the scan of all segments at once.
#include <hip/hip_runtime.h>

#include "gdn_device.h"
#include "gdn_layer.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

template <typename TI, int N, int P>
struct SsmShape {
  static constexpr int S = sizeof(TI);
  static constexpr int GE = 16 / S;                 // elements per 16-byte granule
  static constexpr int C = S == 2 ? 64 : 32;        // tokens per block
  static constexpr int NW = P >= 64 ? 4 : P / 16;   // waves
  static constexpr int THREADS = 64 * NW;
  static constexpr int CW = P / NW;                 // state columns per wave
  static constexpr int CT = CW / 16, RT = C / 16, NT = N / 16;
  static constexpr int TPU = S == 2 ? 2 : 1;        // 16-wide tiles per unit
  static constexpr int NU = (NT + TPU - 1) / TPU;   // units along N
  static constexpr bool HALF = TPU == 2 && NT % 2 == 1;  // N = 16: half a unit
  static constexpr int TU = RT / TPU;               // units along the tokens
  static constexpr int GRB = N / GE, GRX = P / GE;  // granules per row of b (c) and x
  static constexpr int MU = S == 2 ? 6 : 3;         // units of M (row tile it: it / TPU + 1)
  static constexpr int o_b = 0, o_c = C * N * S, o_x = 2 * C * N * S, o_m = o_x + C * P * S;
  static constexpr int o_ml = o_m + MU * 1024;      // M's second terms
  static constexpr int o_w = o_ml + (S == 2 ? MU * 1024 : 0);
  static constexpr int total = o_w + 5 * C * 4;     // cum (two terms), d, w, e
  // first unit of row tile it of M
  static constexpr int mu0(int it) {
    int u = 0;
    for (int i = 0; i < it; ++i) u += i / TPU + 1;
    return u;
  }
};

// Granule g of a row sits at granule g ^ swizzle: the four rows of a lane
// group's transposed read and the 16 rows of an operand read fall on
// distinct banks.
template <int GR>
__device__ __forceinline__ int ssm_swz(int row) {
  return (((row & 3) << 2) | ((row >> 2) & 3)) & (GR < 16 ? GR - 1 : 15);
}

// Waits for this wave's LDS accesses, then for the workgroup (global loads
// and stores stay in flight).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A unit of row `row` of b or c (elements of the 16-wide k-tiles 2u, 2u + 1).
template <typename TI, int GR, bool HALF>
__device__ __forceinline__ typename Unit<TI>::type ssm_row_unit(const char* tile, int row, int u, int q) {
  if constexpr (HALF) {
    const uint2 r = *(const uint2*)(tile + row * GR * 16 + (((q >> 1) ^ ssm_swz<GR>(row)) * 16) + (q & 1) * 8);
    return __builtin_bit_cast(bf16x8, make_uint4(r.x, r.y, 0u, 0u));
  } else {
    return *(const typename Unit<TI>::type*)(tile + row * GR * 16 + (((4 * u + q) ^ ssm_swz<GR>(row)) * 16));
  }
}

// Byte offset in a row of b or c of the four elements 16 nt + 4 k .. + 3.
template <typename TI, int N>
__device__ __forceinline__ int ssm_quad(int row, int nt, int k) {
  constexpr int GR = N * (int)sizeof(TI) / 16;
  if constexpr (sizeof(TI) == 4) return ((4 * nt + k) ^ ssm_swz<GR>(row)) * 16;
  else if constexpr (N == 16) return ((k >> 1) ^ ssm_swz<GR>(row)) * 16 + (k & 1) * 8;
  else return ((4 * (nt >> 1) + k) ^ ssm_swz<GR>(row)) * 16 + (nt & 1) * 8;
}

// The LDS transpose read: lane j of a 16-lane group gets element j % 4 of
// the 8 bytes that lane 4 k + j / 4 names, as its element k.
__device__ __forceinline__ bf16x8 ssm_tr(const char* lo, const char* hi) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)hi);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Column 16 nt + l % 16 of b over the tokens of unit tu (b read transposed).
template <typename TI, int N>
__device__ __forceinline__ typename Unit<TI>::type ssm_b_col(const char* tile, int nt, int tu, int lane) {
  constexpr int RB = N * (int)sizeof(TI);
  const int q = lane >> 4, j = lane & 15;
  if constexpr (sizeof(TI) == 2) {
    const int r = 32 * tu + 4 * q + (j >> 2);
    return ssm_tr(tile + r * RB + ssm_quad<TI, N>(r, nt, j & 3),
                  tile + (r + 16) * RB + ssm_quad<TI, N>(r + 16, nt, j & 3));
  } else {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 16 * tu + 4 * q + e;
      v[e] = *(const float*)(tile + r * RB + ssm_quad<TI, N>(r, nt, j >> 2) + (j & 3) * 4);
    }
    return v;
  }
}

// Column col0 + l % 16 of x over the tokens of unit tu.
template <typename TI, int P>
__device__ __forceinline__ typename Unit<TI>::type ssm_x_col(const char* tile, int col0, int tu, int lane) {
  constexpr int GR = P * (int)sizeof(TI) / 16, RB = P * (int)sizeof(TI);
  const int q = lane >> 4, j = lane & 15;
  if constexpr (sizeof(TI) == 2) {
    const int c = col0 + 4 * (j & 3), g = c >> 3, o = (c & 4) * 2;
    const int r = 32 * tu + 4 * q + (j >> 2);
    return ssm_tr(tile + r * RB + ((g ^ ssm_swz<GR>(r)) * 16) + o,
                  tile + (r + 16) * RB + ((g ^ ssm_swz<GR>(r + 16)) * 16) + o);
  } else {
    const int c = col0 + j;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 16 * tu + 4 * q + e;
      v[e] = *(const float*)(tile + r * RB + (((c >> 2) ^ ssm_swz<GR>(r)) * 16) + (c & 3) * 4);
    }
    return v;
  }
}

// x as two bf16 terms (hi + lo within 2^-17 of it), or as it is.
template <bool HALF>
__device__ __forceinline__ void ssm_split2(const f32x4& t0, const f32x4& t1, bf16x8& hi, bf16x8& lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = (bf16)t0[e];
    lo[e] = (bf16)(t0[e] - (float)hi[e]);
    hi[4 + e] = HALF ? (bf16)0.f : (bf16)t1[e];
    lo[4 + e] = HALF ? (bf16)0.f : (bf16)(t1[e] - (float)hi[4 + e]);
  }
}

__device__ __forceinline__ float ssm_step_size(const float* dt_bias, int h, float dt, int softplus) {
  const float x = dt + (dt_bias ? dt_bias[h] : 0.f);
  if (!softplus) return x;
  return x > 20.f ? x : log1pf(expf(x));
}

// Registers of one block's loads: ROWS rows of GR granules by THREADS threads.
template <int ROWS, int GR, int THREADS>
struct SsmLoad {
  static constexpr int rpi = THREADS / GR;  // rows per pass of the workgroup
  static constexpr int n = (ROWS + rpi - 1) / rpi;
  static_assert(THREADS % GR == 0, "a pass covers whole rows");
  uint4 v[n];
  // rows at or after `rows` read as zeros
  __device__ __forceinline__ void load(const char* base, int64_t stride, int rows, int tid) {
    const int r0 = tid / GR;
    const char* p = base + r0 * stride + (tid % GR) * 16;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + i * rpi < rows) v[i] = ld16(p + i * rpi * stride);
    }
  }
  // in the row's own order
  __device__ __forceinline__ void store(char* tile, int tid) const {
    const int g = tid % GR;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int r = tid / GR + i * rpi;
      if (r < ROWS) st16(tile + r * GR * 16 + ((g ^ ssm_swz<GR>(r)) * 16), v[i]);
    }
  }
  // bf16 rows in k-tile order: the two quads of a granule to their lanes' units
  __device__ __forceinline__ void store_ktile(char* tile, int tid) const {
    const int g = tid % GR, k = 2 * (g & 1), o = ((g >> 1) & 1) * 8, u = (g >> 2) * 4;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int r = tid / GR + i * rpi;
      if (r >= ROWS) continue;
      char* row = tile + r * GR * 16;
      *(uint2*)(row + (((u + k) ^ ssm_swz<GR>(r)) * 16) + o) = make_uint2(v[i].x, v[i].y);
      *(uint2*)(row + (((u + k + 1) ^ ssm_swz<GR>(r)) * 16) + o) = make_uint2(v[i].z, v[i].w);
    }
  }
};

// Where a workgroup's segment lies.
struct SsmSegment {
  int seq, t0, n, slot;
  bool first, last;  // of its sequence
};

__device__ __forceinline__ SsmSegment ssm_segment(const SsmParams& p, int s) {
  SsmSegment g;
  g.slot = s;
  if (p.packed) {
    const int* row = p.table + 4 * (int64_t)s;
    g.seq = row[0];
    g.t0 = row[1];
    g.n = row[2];
    g.first = s == p.seg_off[g.seq];
    g.last = s + 1 == p.seg_off[g.seq + 1];
  } else {
    g.seq = s / p.segs_per_seq;
    const int j = s - g.seq * p.segs_per_seq;
    g.t0 = g.seq * p.seq_len + j * p.seg_len;
    g.n = min(p.seg_len, p.seq_len - j * p.seg_len);
    g.first = j == 0;
    g.last = j + 1 == p.segs_per_seq;
  }
  return g;
}

// Work item of a workgroup: XCD k (workgroups k, k + 8, ...) takes the k-th
// eighth of the items in order, heads fastest, so that the heads that share
// rows of b and c share an L2.
__device__ __forceinline__ int64_t ssm_item(int64_t items) {
  const int64_t per = (items + 7) / 8;
  const int64_t i = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  return (blockIdx.x >> 3) < per && i < items ? i : -1;
}

// OUT: the scan (c, y, states in and out); else a segment's end state.
template <typename TI, int N, int P, bool OUT>
__global__ __launch_bounds__((SsmShape<TI, N, P>::THREADS), 2) void ssm_kernel(SsmParams p) {
  using D = SsmShape<TI, N, P>;
  constexpr int C = D::C, NW = D::NW, CT = D::CT, RT = D::RT, NT = D::NT, NU = D::NU, TU = D::TU;
  constexpr int TPU = D::TPU, S = D::S;
  constexpr bool HALF = D::HALF;
  using U = typename Unit<TI>::type;
  __shared__ __attribute__((aligned(1024))) char smem[D::total];
  char* const sB = smem + D::o_b;
  char* const sC = smem + D::o_c;
  char* const sX = smem + D::o_x;
  char* const sM = smem + D::o_m;
  char* const sL = smem + D::o_ml;
  float* const s_cum = (float*)(smem + D::o_w);
  float* const s_lo = s_cum + C;
  float* const s_d = s_lo + C;
  float* const s_w = s_d + C;
  float* const s_e = s_w + C;

  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t item = ssm_item((int64_t)p.max_segs * p.heads);
  if (item < 0) return;
  const int si = (int)(item / p.heads), h = (int)(item - (int64_t)si * p.heads);
  const int64_t state_elems = (int64_t)N * P;

  if (p.packed && si >= p.seg_off[p.n_seq]) {
    // past the last segment: empty sequences have none, and their state is
    // carried over here (there are at least as many such items as empty
    // sequences)
    if (!OUT || !p.final_state) return;
    const int total = p.seg_off[p.n_seq];
    for (int i = si - total; i < p.n_seq; i += p.max_segs - total) {
      if (p.seg_off[i] != p.seg_off[i + 1]) continue;
      const int64_t o = ((int64_t)i * p.heads + h) * state_elems;
      for (int e = tid; e < state_elems; e += D::THREADS) p.final_state[o + e] = p.init ? p.init[o + e] : 0.f;
    }
    return;
  }
  const SsmSegment sg = ssm_segment(p, si);
  if (!OUT && sg.last) return;  // no later segment needs its end state

  const int grp = h / p.group;
  const int64_t b_st = p.b_st * S, c_st = p.c_st * S, x_st = p.x_st * S;
  const char* pb = (const char*)p.b + sg.t0 * b_st + grp * p.b_sh * S;
  const char* pc = (const char*)p.c + sg.t0 * c_st + grp * p.c_sh * S;
  const char* px = (const char*)p.x + sg.t0 * x_st + h * p.x_sh * S;
  const float* pd = p.dt + sg.t0 * p.dt_st + h * p.dt_sh;
  TI* po = (TI*)p.out + sg.t0 * p.o_st + h * p.o_sh;
  const float rate = -expf(p.a_log ? p.a_log[h] : 0.f) * kLog2e;
  const float skip = OUT && p.d_skip ? p.d_skip[h] : 0.f;
  const int col0 = wave * D::CW;

  SsmLoad<C, D::GRB, D::THREADS> rb, rc;
  SsmLoad<C, D::GRX, D::THREADS> rx;
  float rd = 0.f;
  auto fetch = [&](int t) {
    const int rows = sg.n - t;
    rb.load(pb + t * b_st, b_st, rows, tid);
    if constexpr (OUT) rc.load(pc + t * c_st, c_st, rows, tid);
    rx.load(px + t * x_st, x_st, rows, tid);
    rd = 0.f;
    if (wave == 0 && lane < C && lane < rows) rd = pd[(int64_t)(t + lane) * p.dt_st];
  };
  if (sg.n > 0) fetch(0);

  // the state before the segment: nt, ct tile, lane (q, m) holds rows
  // 16 nt + 4 q + e of column col0 + 16 ct + m
  f32x4 H[NT][CT];
  const int64_t so = ((int64_t)sg.seq * p.heads + h) * state_elems;
  float* slot = p.slots ? p.slots + ((int64_t)sg.slot * p.heads + h) * state_elems : nullptr;
  const int fr = wave * NT * CT * 256 + lane * 4;  // a wave's fragments in a slot
  const bool from_slot = OUT && slot && !(sg.first && sg.last) && !(sg.first && !p.init);
  const float* from = sg.first && !from_slot ? p.init : nullptr;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      H[nt][ct] = zero4();
      if (from_slot) {
        H[nt][ct] = *(const f32x4*)(slot + fr + (nt * CT + ct) * 256);
      } else if (from) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          H[nt][ct][e] = from[so + (int64_t)(16 * nt + 4 * q + e) * P + col0 + 16 * ct + m];
      }
    }
  if (!OUT && sg.first && p.init) {
    // a copy for the scan, which may run beside the write of final_state
    // over the same memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) *(f32x4*)(slot + fr + (nt * CT + ct) * 256) = H[nt][ct];
  }
  float total_log = 0.f;  // the segment's decay so far, base 2

  for (int t = 0; t < sg.n; t += C) {
    lds_barrier();  // the last block's readers are done
    if constexpr (S == 2 && !HALF) {
      rb.store_ktile(sB, tid);
      if constexpr (OUT) rc.store_ktile(sC, tid);
    } else {
      rb.store(sB, tid);
      if constexpr (OUT) rc.store(sC, tid);
    }
    rx.store(sX, tid);
    if (wave == 0) {
      // step sizes and their decays; rows past the end have step 0.  The sum
      // runs in fp64 and is kept as two floats: an fp32 sum of, say, -100
      // would leave 4e-6 in the difference of two neighbours
      const float d = lane < sg.n - t && lane < C ? ssm_step_size(p.dt_bias, h, rd, p.softplus) : 0.f;
      double cum = (double)rate * (double)d;
#pragma unroll
      for (int off = 1; off < C; off <<= 1) {
        const double o = __shfl_up(cum, off);
        if (lane >= off) cum += o;
      }
      const double last = __shfl(cum, C - 1);
      if (lane < C) {
        s_cum[lane] = (float)cum;
        s_lo[lane] = (float)(cum - (double)(float)cum);
        s_d[lane] = d;
        s_w[lane] = d * __builtin_amdgcn_exp2f((float)(last - cum));
        s_e[lane] = __builtin_amdgcn_exp2f((float)cum);
      }
    }
    if (t + C < sg.n) fetch(t + C);
    lds_barrier();
    const float block_log = s_cum[C - 1];
    const float alpha = s_e[C - 1];
    total_log += block_log;

    U xu[TU][CT];  // this wave's columns of x
    if constexpr (OUT) {
      // M's tiles (jt, it), jt <= it, over the waves: transposed products, so
      // that lane (q, m) holds M[16 it + m][16 jt + 4 q + e], an operand's
      // layout
      for (int tile = wave; tile < RT * (RT + 1) / 2; tile += NW) {
        const int it = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0;
        const int jt = tile - it * (it + 1) / 2;
        f32x4 acc = zero4();
#pragma unroll
        for (int u = 0; u < NU; ++u)
          mma_unit<HALF>(acc, ssm_row_unit<TI, D::GRB, HALF>(sB, 16 * jt + m, u, q),
                         ssm_row_unit<TI, D::GRB, HALF>(sC, 16 * it + m, u, q));
        const f32x4 cj = *(const f32x4*)(s_cum + 16 * jt + 4 * q);
        const f32x4 dj = *(const f32x4*)(s_d + 16 * jt + 4 * q);
        const int i = 16 * it + m;
        const f32x4 lj = *(const f32x4*)(s_lo + 16 * jt + 4 * q);
        const float ci = s_cum[i], li = s_lo[i];
        f32x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * jt + 4 * q + e;
          float v = j <= i ? acc[e] * __builtin_amdgcn_exp2f((ci - cj[e]) + (li - lj[e])) * dj[e] : 0.f;
          if (j == i) v += skip;
          hi[e] = v;
          lo[e] = v - to_float(from_float<TI>(v));
        }
        int unit = 0;
#pragma unroll
        for (int i2 = 0; i2 < RT; ++i2)
          if (i2 == it) unit = D::mu0(i2);
        unit += jt / TPU;
        const int o = unit * 1024 + lane * 16 + (TPU == 2 ? (jt & 1) * 8 : 0);
        store4<TI>((TI*)(sM + o), hi[0], hi[1], hi[2], hi[3]);
        if constexpr (S == 2) {
          store4<TI>((TI*)(sL + o), lo[0], lo[1], lo[2], lo[3]);
          if (jt == it && (it & 1) == 0) {  // the unit's second tile lies after the diagonal
            *(uint2*)(sM + o + 8) = make_uint2(0u, 0u);
            *(uint2*)(sL + o + 8) = make_uint2(0u, 0u);
          }
        }
      }

      // y^T tiles: rows are columns of x, columns are tokens
      f32x4 y[RT][CT];
#pragma unroll
      for (int it = 0; it < RT; ++it)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) y[it][ct] = zero4();
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        U cu[RT];
#pragma unroll
        for (int it = 0; it < RT; ++it) cu[it] = ssm_row_unit<TI, D::GRB, HALF>(sC, 16 * it + m, u, q);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          if constexpr (S == 2) {
            bf16x8 hi, lo;
            ssm_split2<HALF>(H[2 * u][ct], H[HALF ? 2 * u : 2 * u + 1][ct], hi, lo);
#pragma unroll
            for (int it = 0; it < RT; ++it) mma_unit<HALF>(y[it][ct], hi, cu[it]);
#pragma unroll
            for (int it = 0; it < RT; ++it) mma_unit<HALF>(y[it][ct], lo, cu[it]);
          } else {
#pragma unroll
            for (int it = 0; it < RT; ++it) mma_unit<HALF>(y[it][ct], H[u][ct], cu[it]);
          }
        }
      }
#pragma unroll
      for (int it = 0; it < RT; ++it) {
        const float e = s_e[16 * it + m];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[it][ct][r] *= e;
      }
#pragma unroll
      for (int tu = 0; tu < TU; ++tu)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) xu[tu][ct] = ssm_x_col<TI, P>(sX, col0 + 16 * ct, tu, lane);
      lds_barrier();  // M is complete
#pragma unroll
      for (int it = 0; it < RT; ++it)
#pragma unroll
        for (int ju = 0; ju <= it / TPU; ++ju) {
          const int o = (D::mu0(it) + ju) * 1024 + lane * 16;
          const U mh = *(const U*)(sM + o);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(y[it][ct], xu[ju][ct], mh);
          if constexpr (S == 2) {
            const U ml = *(const U*)(sL + o);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) mma_unit<false>(y[it][ct], xu[ju][ct], ml);
          }
        }
#pragma unroll
      for (int it = 0; it < RT; ++it) {
        const int i = t + 16 * it + m;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          settle(y[it][ct]);
          if (i < sg.n)
            store4<TI>(po + (int64_t)i * p.o_st + col0 + 16 * ct + 4 * q, y[it][ct][0], y[it][ct][1],
                       y[it][ct][2], y[it][ct][3]);
        }
      }
    } else {
#pragma unroll
      for (int tu = 0; tu < TU; ++tu)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) xu[tu][ct] = ssm_x_col<TI, P>(sX, col0 + 16 * ct, tu, lane);
    }

    // the state update
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[nt][ct][e] *= alpha;
#pragma unroll
    for (int tu = 0; tu < TU; ++tu) {
      if constexpr (S == 2) {
        const f32x4 w0 = *(const f32x4*)(s_w + 32 * tu + 4 * q);
        const f32x4 w1 = *(const f32x4*)(s_w + 32 * tu + 16 + 4 * q);
        bf16x8 a0[CT], a1[CT], a2[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = (float)xu[tu][ct][e] * (e < 4 ? w0[e & 3] : w1[e & 3]);
            a0[ct][e] = (bf16)v;
            const float r = v - (float)a0[ct][e];
            a1[ct][e] = (bf16)r;
            a2[ct][e] = (bf16)(r - (float)a1[ct][e]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const U b = ssm_b_col<TI, N>(sB, nt, tu, lane);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a0[ct]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a1[ct]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a2[ct]);
        }
      } else {
        const f32x4 w = *(const f32x4*)(s_w + 16 * tu + 4 * q);
        f32x4 a[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e) a[ct][e] = xu[tu][ct][e] * w[e];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const U b = ssm_b_col<TI, N>(sB, nt, tu, lane);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a[ct]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) settle(H[nt][ct]);
  }

  if constexpr (OUT) {
    if (sg.last && p.final_state) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p.final_state[so + (int64_t)(16 * nt + 4 * q + e) * P + col0 + 16 * ct + m] = H[nt][ct][e];
    }
  } else {
    // into the next segment's slot
    float* dst = slot + (int64_t)p.heads * state_elems;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) *(f32x4*)(dst + fr + (nt * CT + ct) * 256) = H[nt][ct];
    if (tid == 0) p.seg_decay[(int64_t)sg.slot * p.heads + h] = __builtin_amdgcn_exp2f(total_log);
  }
}

// Joins a sequence's segments: the state before segment s is its
// predecessor's end state plus the predecessor's decay times the state before
// that one.  One thread per four elements of a (sequence, head) state.
constexpr int kSsmJoinThreads = 256;

__global__ __launch_bounds__(kSsmJoinThreads) void ssm_join_kernel(SsmParams p, int vecs) {
  const int64_t u = (int64_t)blockIdx.x * kSsmJoinThreads + threadIdx.x;
  const int64_t unit = u / vecs;
  if (unit >= (int64_t)p.n_seq * p.heads) return;
  const int seq = (int)(unit / p.heads), h = (int)(unit - (int64_t)seq * p.heads);
  const int s0 = p.packed ? p.seg_off[seq] : seq * p.segs_per_seq;
  const int s1 = p.packed ? p.seg_off[seq + 1] : s0 + p.segs_per_seq;
  if (s1 - s0 < 3) return;
  const int64_t step = (int64_t)p.heads * vecs;
  f32x4* v = (f32x4*)p.slots + ((int64_t)(s0 + 1) * p.heads + h) * vecs + (u - unit * vecs);
  const float* dec = p.seg_decay + (int64_t)(s0 + 1) * p.heads + h;
  f32x4 carry = *v;
  for (int s = s0 + 2; s < s1; ++s) {
    v += step;
    const f32x4 e = *v;
    const float d = *dec;
    dec += p.heads;
#pragma unroll
    for (int i = 0; i < 4; ++i) carry[i] = e[i] + d * carry[i];
    *v = carry;
  }
}

// ---------------------------------------------------------------------------
// One token per sequence: reads and writes the state once, so it is bound by
// HBM.  A workgroup takes CB columns of one head's state; each thread holds
// four adjacent columns of a band of rows, read and written with 16-byte
// accesses; the contraction with c is reduced over the bands through LDS.

template <int N, int P>
struct SsmStepShape {
  static constexpr int CB = P < 32 ? P : 32;          // columns per workgroup
  static constexpr int CG = CB / 4;                   // column groups
  static constexpr int RG = N < 256 / CG ? N : 256 / CG;  // row groups
  static constexpr int NT = CG * RG;
  static constexpr int RPT = N / RG;
};

template <typename TI, int N, int P>
__global__ __launch_bounds__((SsmStepShape<N, P>::NT)) void ssm_step_kernel(SsmStepParams p) {
  using D = SsmStepShape<N, P>;
  constexpr int CB = D::CB, CG = D::CG, RG = D::RG, RPT = D::RPT;
  __shared__ __attribute__((aligned(16))) float sred[RG][CB];
  constexpr int SL = P / CB;
  const int u = blockIdx.x / SL, sl = blockIdx.x % SL;
  const int i = u / p.heads, h = u - i * p.heads, grp = h / p.group;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int c0 = sl * CB + 4 * cg, r0 = rg * RPT;
  float* Hs = p.state + ((int64_t)u * N + r0) * P + c0;
  f32x4 hreg[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) hreg[r] = *(const f32x4*)(Hs + r * P);
  const TI* br = (const TI*)p.b + (int64_t)i * p.b_st + (int64_t)grp * p.b_sh + r0;
  const TI* cr = (const TI*)p.c + (int64_t)i * p.c_st + (int64_t)grp * p.c_sh + r0;
  const f32x4 x = load4<TI>((const TI*)p.x + (int64_t)i * p.x_st + (int64_t)h * p.x_sh + c0);
  const float d = ssm_step_size(p.dt_bias, h, p.dt[(int64_t)i * p.dt_st + (int64_t)h * p.dt_sh], p.softplus);
  const float a = expf(-expf(p.a_log ? p.a_log[h] : 0.f) * d);
  f32x4 part = zero4();
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const float bv = d * to_float(br[r]), cv = to_float(cr[r]);
    f32x4 hn;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hn[e] = a * hreg[r][e] + bv * x[e];
      part[e] += cv * hn[e];
    }
    *(f32x4*)(Hs + r * P) = hn;
  }
  *(f32x4*)&sred[rg][4 * cg] = part;
  __syncthreads();
  if (rg == 0) {
    f32x4 o = zero4();
    for (int k = 0; k < RG; ++k) {
      const f32x4 t = *(const f32x4*)&sred[k][4 * cg];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += t[e];
    }
    const float skip = p.d_skip ? p.d_skip[h] : 0.f;
    store4<TI>((TI*)p.out + (int64_t)i * p.o_st + (int64_t)h * p.o_sh + c0, o[0] + skip * x[0],
               o[1] + skip * x[1], o[2] + skip * x[2], o[3] + skip * x[3]);
  }
}

// ---------------------------------------------------------------------------
// dispatch

int ssm_target_groups() { return 512; }

template <typename TI, int N, int P>
static hipError_t launch_ssm_np(bool out, const SsmParams& p, hipStream_t s) {
  const int64_t items = (int64_t)p.max_segs * p.heads, blocks = (items + 7) / 8 * 8;
  if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), threads(SsmShape<TI, N, P>::THREADS);
  if (out) {
    hipLaunchKernelGGL((ssm_kernel<TI, N, P, true>), grid, threads, 0, s, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((ssm_kernel<TI, N, P, false>), grid, threads, 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.packed && p.segs_per_seq < 3)) return e;
  const int vecs = N * P / 4;
  const int64_t join = ((int64_t)p.n_seq * p.heads * vecs + kSsmJoinThreads - 1) / kSsmJoinThreads;
  if (join >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)join), dim3(kSsmJoinThreads), 0, s, p, vecs);
  return hipGetLastError();
}

template <typename TI, int N, int P>
static hipError_t launch_ssm_step_np(const SsmStepParams& p, hipStream_t s) {
  using D = SsmStepShape<N, P>;
  const int64_t blocks = (int64_t)p.n * p.heads * (P / D::CB);
  if (blocks >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ssm_step_kernel<TI, N, P>), dim3((unsigned)blocks), dim3(D::NT), 0, s, p);
  return hipGetLastError();
}

#define GDN_SSM_SIZES(X) \
  X(16, 16) X(16, 32) X(16, 64) X(16, 128) X(32, 16) X(32, 32) X(32, 64) X(32, 128) \
  X(64, 16) X(64, 32) X(64, 64) X(64, 128) X(128, 16) X(128, 32) X(128, 64) X(128, 128)

static hipError_t launch_ssm(bool bf16, int n, int pp, bool out, const SsmParams& sp, hipStream_t s) {
#define GDN_X(NN, PP)        \
  if (n == NN && pp == PP)   \
    return bf16 ? launch_ssm_np<gdn::bf16, NN, PP>(out, sp, s) : launch_ssm_np<float, NN, PP>(out, sp, s);
  GDN_SSM_SIZES(GDN_X)
#undef GDN_X
  return hipErrorInvalidValue;
}

hipError_t launch_ssm_states(bool bf16, int n, int p, const SsmParams& sp, hipStream_t s) {
  return launch_ssm(bf16, n, p, false, sp, s);
}
hipError_t launch_ssm_scan(bool bf16, int n, int p, const SsmParams& sp, hipStream_t s) {
  return launch_ssm(bf16, n, p, true, sp, s);
}

hipError_t launch_ssm_step(bool bf16, int n, int p, const SsmStepParams& sp, hipStream_t s) {
#define GDN_X(NN, PP)       \
  if (n == NN && p == PP)   \
    return bf16 ? launch_ssm_step_np<gdn::bf16, NN, PP>(sp, s) : launch_ssm_step_np<float, NN, PP>(sp, s);
  GDN_SSM_SIZES(GDN_X)
#undef GDN_X
  return hipErrorInvalidValue;
}

}  // namespace gdn
