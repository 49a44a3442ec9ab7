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
// and S; 2^-16 of a product, below the output's own rounding), three for the
// state where it is handed on (w_t x_t; 2^-24, so the fp32 state keeps fp32
// accuracy) and two where only this segment's outputs read it: bf16 outputs
// differ from those of fp32 products in 1e-4 (their own rounding: 1.7e-3).
// fp32 inputs use fp32 matrix instructions throughout (1.3e-7 from 64 bits, as
// a plain fp32 evaluation).  Sums of steps are run in fp64.
//
// A workgroup of eight waves scans one segment of one 128-column head or of
// two 64-column ones (fewer waves for fewer columns), in blocks of C = 32
// tokens, the state in the accumulators of its waves (each wave holds all N
// rows of 16 columns).  The fragment layout along the contraction index is
// the accumulators' own, so the state and x feed the products without leaving
// their lanes; b, c and x lie in LDS as in memory (granules swizzled), and
// what meets the token axis is read transposed.  All waves copy the tiles of
// the coming blocks straight to LDS, b and c two blocks ahead (the next
// block's M is formed beside this block's products, so that a block needs one
// barrier), x one.
//
// A sequence cut into segments takes three launches: the segments' end
// states from zero (the same kernel without c and y), their joining in
// order, and the scan of all segments at once.
//
// What bounds it: not the bytes (16384 tokens x 48 heads of 128 x 128 in
// bf16: 546 MB in 294 us, 288 to 306 over several cards, 1.9 TB/s) nor LDS
// (45 % busy; tiles laid out with half the bank conflicts took as long), but
// issue.  A wave issues about 256 vector instructions and 38 matrix ones a
// block, 96 of the former to split the state into terms; a matrix instruction
// of 16 cycles lets two vector instructions of other waves in where four would
// fit (both measured), so the two together take about 75 % of a SIMD's cycles
// (counters: vector unit 62 %, matrix cores 32 %), and the block's barrier the
// rest.  Two blocks a barrier for the segments' states and batched joining
// took that case from 305 to 291 us when they were built.  No faster: copies by
// a ninth wave, ageing the state less often, raised priority for the matrix
// phases, deeper rings, the split by dot products (they take the matrix unit's
// slots).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_layer.h"
#include "gdn_tiles.h"

namespace gdn {

// HP: heads (of one group) that a workgroup takes.
template <typename TI, int N, int P, int HP, bool OUT>
struct SsmShape {
  static constexpr int S = sizeof(TI);
  static constexpr int C = 32;                      // tokens per block
  static constexpr int CW = 16;                     // state columns per wave
  static constexpr int NH = P / CW, NW = NH * HP;   // waves of a head, of all
  static constexpr int THREADS = 64 * NW;
  static constexpr int CT = CW / 16, RT = C / 16, NT = N / 16;
  static constexpr int TPU = S == 2 ? 2 : 1;        // 16-wide tiles per unit
  static constexpr int NU = (NT + TPU - 1) / TPU;   // units along N
  static constexpr bool HALF = TPU == 2 && NT % 2 == 1;  // N = 16: half a unit
  static constexpr int TU = RT / TPU;               // units along the tokens
  static constexpr int TILES = RT * (RT + 1) / 2;   // of M
  // LDS: rings of b (and c), of x, of the blocks' weights (and, for M, which
  // is a block ahead, of its sums and steps), and M's two buffers
  static constexpr int BB = C * N * S, XB = C * P * S, MB = 3072, WB = 2 * C * 4, GB = OUT ? 2 * C * 4 + C * 2 : 0;
  static constexpr int RB = OUT ? 3 : 4, RX = OUT ? 2 : 4, RW = 4, RG = RB;
  static constexpr int bc = BB * (OUT ? 2 : 1);     // b, then c
  // (each head has its own x, M and decays)
  static constexpr int o_x = RB * bc, o_m = o_x + HP * RX * XB, o_w = o_m + (OUT ? HP * 2 * MB : 0);
  static constexpr int o_g = o_w + HP * RW * WB, total = o_g + HP * RG * GB;
};

// First row of lane group q's four rows of state tile nt.  bf16 pairs the
// tiles (2u, 2u + 1) so that a lane's rows of the pair are eight consecutive
// ones, the granule of a row of b or c that it meets.
template <typename TI, int N>
__device__ __forceinline__ int ssm_state_row(int nt, int q) {
  if (sizeof(TI) == 2 && N >= 32) return 32 * (nt >> 1) + 8 * q + 4 * (nt & 1);
  return 16 * nt + 4 * q;
}

// Operand reads from the tiles.  Everything but the lane's own place is a
// compile-time constant: rows 16 apart have the same swizzle, and unit u of a
// row differs from unit 0 by an exclusive or in the granule's upper bits.
template <typename TI, int N>
struct SsmRows {
  static constexpr int RB = N * (int)sizeof(TI), GR = RB / 16;
  static constexpr bool HALF = RB == 32;  // bf16, N = 16: half a unit
  uint32_t row;  // of unit 0 of row l % 16
  uint32_t col;  // of the transposed read's first quad, column tile 0
  __device__ __forceinline__ SsmRows(int lane) {
    const int q = lane >> 4, m = lane & 15, k = lane & 3, r = 4 * q + ((lane >> 2) & 3);
    if constexpr (HALF) {
      row = m * RB + (((q >> 1) ^ ssm_swz<GR>(m)) * 16) + (q & 1) * 8;
      col = r * RB + (((k >> 1) ^ ssm_swz<GR>(r)) * 16) + (k & 1) * 8;
    } else {
      row = m * RB + ((q ^ ssm_swz<GR>(m)) * 16);
      col = r * RB + ((k ^ ssm_swz<GR>(r)) * 16);
    }
  }
  // unit u of row 16 it + l % 16 (`it` may be a run-time value)
  __device__ __forceinline__ typename Unit<TI>::type unit(const char* tile, int it, int u) const {
    if constexpr (HALF) {
      const uint2 r = *(const uint2*)(tile + row + it * 16 * RB);
      return __builtin_bit_cast(bf16x8, make_uint4(r.x, r.y, 0u, 0u));
    } else {
      return *(const typename Unit<TI>::type*)(tile + (row ^ (u * 64)) + it * 16 * RB);
    }
  }
  // column 16 nt + l % 16 over the tokens of unit tu
  __device__ __forceinline__ typename Unit<TI>::type column(const char* tile, int nt, int tu, int lane) const;
};

template <typename TI, int N>
__device__ __forceinline__ typename Unit<TI>::type SsmRows<TI, N>::column(const char* tile, int nt, int tu,
                                                                         int lane) const {
  if constexpr (sizeof(TI) == 2) {
    const char* a = tile + (col ^ ((nt >> 1) * 64)) + (nt & 1) * 8 + tu * 32 * RB;
    return ssm_tr(a, a + 16 * RB);
  } else {
    const int q = lane >> 4, j = lane & 15;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * q + e;
      v[e] = *(const float*)(tile + ((r * RB + (((j >> 2) ^ ssm_swz<GR>(r)) * 16) + (j & 3) * 4) ^ (nt * 64)) +
                             tu * 16 * RB);
    }
    return v;
  }
}

__device__ __forceinline__ float ssm_step_size(float bias, float dt, int softplus) {
  const float x = dt + bias;
  if (!softplus) return x;
  return x > 20.f ? x : log1pf(expf(x));
}

// -scale e^a_log, held above minus infinity, so that a step of zero still
// keeps all memory.
__device__ __forceinline__ float ssm_rate(const float* a_log, int h, float scale) {
  const float r = -expf(a_log ? a_log[h] : 0.f) * scale;
  return r < -0x1.fffffep127f ? -0x1.fffffep127f : r;
}

typedef unsigned int ssm_u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int ssm_u32x4 __attribute__((ext_vector_type(4)));

// A block's rows of one tensor, from its first row on: accesses past the last
// row's end read zeros and write nothing (the hardware's range check).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t ssm_rows(const void* base, int64_t stride, int rows, int row_bytes) {
  const uint32_t bytes = rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)stride + (uint32_t)row_bytes : 0u;
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, 0x00027000);
}

template <typename TI>
__device__ __forceinline__ void ssm_store4(__amdgpu_buffer_rsrc_t r, uint32_t offset, const f32x4& a) {
  typename Quad<TI>::type v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = from_float<TI>(a[e]);
  if constexpr (sizeof(TI) == 2)
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(ssm_u32x2, v), r, (int)offset, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(ssm_u32x4, v), r, (int)offset, 0, 0);
}

template <int V>
struct SsmInt {
  static constexpr int value = V;
};

// Copies a block's rows of one tensor into a tile, granules swizzled (rows at
// or after `rows` as zeros), straight to LDS, 1 KiB pieces over the waves.
// Written as assembly so that the compiler does not wait for the copies at
// every LDS read; the wave waits for them itself before the barrier that
// hands them over.
template <int ROWS, int GR, int NW>
struct SsmCopy {
  static constexpr int pieces = ROWS * GR / 64;
  static constexpr int n = (pieces + NW - 1) / NW;  // a wave's, the last ones repeated
  __device__ __forceinline__ static void issue(uint32_t tile, const char* base, int64_t stride, int rows, int wave,
                                               int lane) {
    rows = min(rows, ROWS);
    ssm_u32x4 words;  // the buffer descriptor of ssm_rows
    words[0] = (uint32_t)(uintptr_t)base;
    words[1] = (uint32_t)((uintptr_t)base >> 32) & 0xffffu;
    words[2] = rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)stride + (uint32_t)(GR * 16) : 0u;
    words[3] = 0x00027000u;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int piece = min(wave + i * NW, pieces - 1);
      const int g = piece * 64 + lane, row = g / GR;
      const uint32_t o = (uint32_t)row * (uint32_t)stride + (uint32_t)((g % GR) ^ ssm_swz<GR>(row)) * 16u;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                   :
                   : "s"(__builtin_amdgcn_readfirstlane(tile + piece * 1024)), "v"(o), "s"(words)
                   : "memory", "m0");
    }
  }
};

// Where a workgroup's segment lies.
struct SsmSegment {
  int seq, t0, n, slot;  // slot < 0: the sequence is not cut
  bool first, last;  // of its sequence
};

template <bool OUT>
__device__ __forceinline__ SsmSegment ssm_segment(const SsmParams& p, int s) {
  SsmSegment g;
  if (p.packed) {
    const int4 row = *(const int4*)((OUT ? p.table : p.cut_table) + 4 * (int64_t)s);
    g.seq = row.x;
    g.t0 = row.y;
    g.n = row.z;
    g.slot = row.w >> 2;
    g.first = row.w & 1;
    g.last = row.w & 2;
  } else {
    g.seq = s / p.segs_per_seq;
    const int j = s - g.seq * p.segs_per_seq;
    g.slot = p.segs_per_seq > 1 ? s + g.seq : -1;
    g.t0 = g.seq * p.seq_len + j * p.seg_len;
    g.n = min(p.seg_len, p.seq_len - j * p.seg_len);
    g.first = j == 0;
    g.last = j + 1 == p.segs_per_seq;
  }
  return g;
}

// A workgroup's segment and first head.  Workgroups k, k + 8, ... run on one
// XCD: a unit of heads of one group and segment, which read the same rows of
// b and c, goes to one of them (one L2), and the units go round them, so that
// each has its share whatever number of the segments is real.
struct SsmItem {
  int seg, head;  // seg < 0: none
};

__device__ __forceinline__ SsmItem ssm_item(const SsmParams& p, int hp) {
  const int hu = p.unit / hp, per_seg = p.heads / p.unit;  // workgroups of a unit, units of a segment
  const int i = blockIdx.x >> 3;
  const int64_t unit = (int64_t)(i / hu) * 8 + (blockIdx.x & 7);
  SsmItem it;
  it.seg = unit < (int64_t)p.max_segs * per_seg ? (int)(unit / per_seg) : -1;
  it.head = (int)(unit % per_seg) * p.unit + (i % hu) * hp;
  return it;
}

// OUT: the scan (c, y, states in and out); else a segment's end state.
template <typename TI, int N, int P, int HP, bool OUT>
__global__ __launch_bounds__((SsmShape<TI, N, P, HP, OUT>::THREADS), (sizeof(TI) == 2 ? 4 : 2)) void ssm_kernel(SsmParams p) {
  using D = SsmShape<TI, N, P, HP, OUT>;
  constexpr int C = D::C, NW = D::NW, NH = D::NH, CT = D::CT, RT = D::RT, NT = D::NT, NU = D::NU, TU = D::TU;
  constexpr int TPU = D::TPU, S = D::S;
  constexpr bool HALF = D::HALF;
  using U = typename Unit<TI>::type;
  __shared__ __attribute__((aligned(1024))) char smem[D::total];

  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const SsmItem item = ssm_item(p, HP);
  if (item.seg < 0) return;
  const int si = item.seg;
  const int hh = wave / NH, wh = wave - hh * NH;  // the wave's head here, and its place in the head
  const int h = item.head + hh;
  const int64_t state_elems = (int64_t)N * P;

  if (!OUT && p.packed && si >= p.cuts[1]) return;  // past the last cut segment
  if (OUT && p.packed && si >= p.seg_off[p.n_seq]) {
    // past the last segment: empty sequences have none, and their state is
    // carried over here (there are at least as many such items as empty
    // sequences)
    if (!p.final_state) return;
    const int total = p.seg_off[p.n_seq];
    for (int i = si - total; i < p.n_seq; i += p.max_segs - total) {
      if (p.seg_off[i] != p.seg_off[i + 1]) continue;
      const int64_t o = ((int64_t)i * p.heads + h) * state_elems;
      for (int e = tid - hh * 64 * NH; e < state_elems; e += 64 * NH) p.final_state[o + e] = p.init ? p.init[o + e] : 0.f;
    }
    return;
  }
  const SsmSegment sg = ssm_segment<OUT>(p, si);
  // a last segment's end state is needed only for the final state
  if (!OUT && sg.last && !p.final_state) return;
  const int blocks = (sg.n + C - 1) / C;
  // The copies: each turn asks for what the next turn needs (b and c two
  // blocks ahead, since the next block's M is formed a block ahead; x one).
  const int grp = h / p.group;
  const int64_t b_st = p.b_st * S, c_st = p.c_st * S, x_st = p.x_st * S, d_st = p.dt_st * 4;
  const char* pb = (const char*)p.b + sg.t0 * b_st + grp * p.b_sh * S;
  const char* pc = OUT ? (const char*)p.c + sg.t0 * c_st + grp * p.c_sh * S : nullptr;
  const char* px = (const char*)p.x + sg.t0 * x_st + h * p.x_sh * S;
  const char* pd = (const char*)(p.dt + sg.t0 * p.dt_st + h * p.dt_sh);
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  auto copy_bc = [&](int blk, int ring) {
    const int t = blk * C;
    SsmCopy<C, N * S / 16, NW>::issue(lds + ring * D::bc, pb + t * b_st, b_st, sg.n - t, wave, lane);
    if constexpr (OUT)
      SsmCopy<C, N * S / 16, NW>::issue(lds + ring * D::bc + D::BB, pc + t * c_st, c_st, sg.n - t, wave, lane);
  };
  auto copy_x = [&](int blk, int ring) {
    const int t = blk * C;
    SsmCopy<C, P * S / 16, NH>::issue(lds + D::o_x + (ring * HP + hh) * D::XB, px + t * x_st, x_st, sg.n - t, wh, lane);
  };
  // raw steps of blocks blk and blk + 1, one token a lane
  auto fetch_steps = [&](int blk) {
    const int t = blk * C;
    const __amdgpu_buffer_rsrc_t r = ssm_rows(pd + t * d_st, d_st, min(sg.n - t, 2 * C), 4);
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)((uint32_t)lane * (uint32_t)d_st), 0, 0));
  };
  const float rate = ssm_rate(p.a_log, h, kLog2e);
  const float bias = p.dt_bias ? p.dt_bias[h] : 0.f;
  // Steps d and decays of blocks blk and blk + 1 (tokens past the end have
  // step 0).  In logarithms to base 2:
  //   c  sum of the token's own tile of 16 up to it,   E = 2^c,
  //   f  d 2^(the tile's sum - c)
  // The sum is run in fp64, and M, which needs its differences, gets it as a
  // float and its remainder: one large step leaves a sum of, say, -1000 for
  // the rest of the tile, of which a float alone would leave 3e-5 in the
  // difference of two neighbours.  A decay past 2^-160 is zero in fp32 and so
  // is every sum that it is part of; held there, sums end at -2560, with
  // remainders below 2^-13, which 2^12 brings into the fp16 range.
  auto weigh = [&](int blk, float raw, int g0, int g1) {
    const float d = blk * C + lane < sg.n ? ssm_step_size(bias, raw, p.softplus) : 0.f;
    double c = (double)rate * (double)d;
    c = c < -160. ? -160. : c;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const double o = __shfl_up(c, off, 16);
      if ((lane & 15) >= off) c += o;
    }
    const double end = __shfl(c, 15, 16);
    float* w = (float*)(smem + D::o_w + (((blk + (lane >> 5)) & (D::RW - 1)) * HP + hh) * D::WB) + (lane & 31);
    w[0] = d * __builtin_amdgcn_exp2f((float)(end - c));
    w[C] = __builtin_amdgcn_exp2f((float)c);
    if constexpr (OUT) {
      char* g = smem + D::o_g + (g0 * HP + hh) * D::GB + (lane >> 5) * ((g1 - g0) * HP * D::GB);
      float* s = (float*)g + (lane & 31);
      s[0] = (float)c;
      s[C] = d;
      ((_Float16*)(g + 8 * C))[lane & 31] = (_Float16)((float)(c - (double)(float)c) * 0x1p12f);
    }
  };
  copy_bc(0, 0);
  copy_bc(1, 1);
  copy_x(0, 0);
  if constexpr (!OUT) copy_x(1, 1);
  // Pairs of blocks are weighed in turn by the waves of the SIMD that has the
  // least of M to form (the fourth one's none of its three tiles; 64 prompts x
  // 16 heads of 64 columns: 327 us, 341 with all waves in turn), without M by
  // all waves.
  constexpr int LAST = OUT ? std::min(NH, 4) - 1 : 0, WN = NH / (LAST + 1);
  const int turn = (wh & LAST) == LAST ? wh >> (LAST == 3 ? 2 : LAST) : -1;
  float raw = turn >= 0 ? fetch_steps(2 * turn) : 0.f;

  // The state before the segment.  Tile (nt, ct), lane (q, m), element e:
  // row ssm_state_row(nt, q) + e, column col0 + 16 ct + m.
  const int col0 = wh * D::CW;
  f32x4 H[NT][CT];
  const int64_t so = ((int64_t)sg.seq * p.heads + h) * state_elems;
  float* slot = sg.slot >= 0 ? p.slots + ((int64_t)sg.slot * p.heads + h) * state_elems : nullptr;
  const int fr = wh * NT * CT * 256 + lane * 4;  // a wave's fragments in a slot
  const bool from_slot = OUT && slot && !(sg.first && !p.init);
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
          H[nt][ct][e] = from[so + (int64_t)(ssm_state_row<TI, N>(nt, q) + e) * P + col0 + 16 * ct + m];
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
  float skip = OUT && p.d_skip ? p.d_skip[h] : 0.f;
  asm volatile("" : "+v"(skip));  // loaded here, not inside the loop
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) settle(H[nt][ct]);
  // a state that is handed on takes three terms, one that only this segment
  // reads two (of a sequence's only segment, whether or not the final state is
  // asked for: its outputs are the same)
  const bool third = !OUT || (sg.first && sg.last);
  SsmRows<TI, N> rows(lane);
  SsmCols<TI, P> cols(col0, lane);
  uint32_t l8 = lane * 8;
  const int64_t o_st = p.o_st * S;
  char* po = (char*)p.out + sg.t0 * o_st + h * p.o_sh * S;
  float decay = 1.f;  // the segment's so far
  asm volatile("" : "+v"(l8));

  // M of a block: transposed products, so that lane (q, m) holds M[16 it + m]
  // [16 jt + 4 q + e], an operand's layout; one tile (0,0), (1,0), (1,1) a wave.
  // bf16: the two terms of tile (0,0) as half units at 0 and 1536, of (1, jt)
  // as the halves of full units at 512 and 2048; fp32: a unit per tile.
  auto form_m = [&](const char* sB, const float* w, const char* g, char* sM) {
    const int q = l8 >> 7, m = (l8 >> 3) & 15;
#pragma unroll 1
    for (int tile = wh; tile < D::TILES; tile += NH) {
      const int it = tile > 0, jt = tile > 1;
      f32x4 acc = zero4();
#pragma unroll
      for (int u = 0; u < NU; ++u) mma_unit<HALF>(acc, rows.unit(sB, jt, u), rows.unit(sB + D::BB, it, u));
      f32x4 v;
      if (it == jt) {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        const float* s = (const float*)g;
        const _Float16* rest = (const _Float16*)(g + 8 * C);
        const f32x4 cj = *(const f32x4*)(s + 16 * jt + 4 * q), dj = *(const f32x4*)(s + C + 16 * jt + 4 * q);
        const f16x4 rj = *(const f16x4*)(rest + 16 * jt + 4 * q);
        const float ci = s[16 * it + m], ri = (float)rest[16 * it + m] * 0x1p-12f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 4 * q + e;
          const float diff = (ci - cj[e]) + __builtin_fmaf((float)rj[e], -0x1p-12f, ri);
          v[e] = acc[e] * (__builtin_amdgcn_exp2f(j <= m ? diff : -__builtin_inff()) * dj[e]) +
                 (j == m ? skip : 0.f);
        }
      } else {
        // through the end of column tile 0, which lies between j and i
        const f32x4 fj = *(const f32x4*)(w + 4 * q);
        const float ei = w[C + 16 + m];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[e] * fj[e] * ei;
      }
      settle(v);
      if constexpr (S == 4) {
        *(f32x4*)(sM + tile * 1024 + l8 * 2) = v;
      } else {
        uint32_t p0[2], p1[2];
        ssm_terms<2>(v[0], v[1], p0);
        ssm_terms<2>(v[2], v[3], p1);
        char* dst = sM + (it == 0 ? l8 : 512 + l8 * 2 + jt * 8);
        *(uint2*)dst = make_uint2(p0[0], p1[0]);
        *(uint2*)(dst + 1536) = make_uint2(p0[1], p1[1]);
      }
    }
  };

  if (turn == 0) {
    weigh(0, raw, 0, 1);
    raw = fetch_steps(2 * WN);
  }
  int rb = 0, rx = 0;
  __builtin_amdgcn_s_waitcnt(ssm_vmcnt(0));  // (the copies, the raw steps)
  if constexpr (OUT) {
    lds_barrier();
    form_m(smem, (const float*)(smem + D::o_w + hh * D::WB), smem + D::o_g + hh * D::GB, smem + D::o_m + hh * D::MB);
  }
  for (int t = 0; t < blocks; ++t) {
    if constexpr (OUT) {
      // the last turn's copies have landed: only its stores are younger
      __builtin_amdgcn_s_waitcnt(ssm_vmcnt(RT * CT));
      lds_barrier();
      copy_bc(t + 2, rb == 0 ? 2 : rb - 1);
      copy_x(t + 1, rx ^ 1);
    } else if ((t & 1) == 0) {
      // two blocks a turn
      __builtin_amdgcn_s_waitcnt(ssm_vmcnt(0));
      lds_barrier();
      copy_bc(t + 2, rb ^ 2);
      copy_x(t + 2, rx ^ 2);
      copy_bc(t + 3, rb ^ 3);
      copy_x(t + 3, rx ^ 3);
    }
    if ((t & 1) == 0 && ((t >> 1) + 1) % WN == turn) {
      weigh(t + 2, raw, rb == 0 ? 2 : rb - 1, rb);  // (a turn back is two on in a ring of three)
      raw = fetch_steps(t + 2 + 2 * WN);
    }
    // the places in the tiles, kept as they are: addresses derived from them
    // outside the loop would take more registers than there are
    asm volatile("" : "+v"(rows.row), "+v"(rows.col), "+v"(cols.at[0]), "+v"(l8));
    const int q = l8 >> 7, m = (l8 >> 3) & 15;
    const char* sB = smem + rb * D::bc;
    const char* sX = smem + D::o_x + (rx * HP + hh) * D::XB;
    const float* w = (const float*)(smem + D::o_w + ((t & (D::RW - 1)) * HP + hh) * D::WB);
    rb = rb + 1 == D::RB ? 0 : rb + 1;
    rx = rx + 1 == D::RX ? 0 : rx + 1;
    const float e0 = w[C + 15], e1 = w[C + 31];
    const float alpha = e0 * e1;
    decay *= alpha;
    U xu[TU][CT];  // this wave's columns of x
#pragma unroll
    for (int tu = 0; tu < TU; ++tu)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) xu[tu][ct] = cols.column(sX, ct, tu);
    if constexpr (OUT) {
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
        for (int it = 0; it < RT; ++it) cu[it] = rows.unit(sB + D::BB, it, u);
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
        const float e = it == 0 ? w[C + m] : w[C + 16 + m] * e0;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) y[it][ct][r] *= e;
      }
      const char* sM = smem + D::o_m + ((t & 1) * HP + hh) * D::MB;
      if constexpr (S == 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint2 a = *(const uint2*)(sM + k * 1536 + l8);
          const U m0 = __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, 0u, 0u));
          const U m1 = *(const U*)(sM + k * 1536 + 512 + l8 * 2);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            mma_unit<true>(y[0][ct], xu[0][ct], m0);
            mma_unit<false>(y[1][ct], xu[0][ct], m1);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          const U mk = *(const U*)(sM + k * 1024 + l8 * 2);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) mma_unit<false>(y[k > 0][ct], xu[k > 1 ? TU - 1 : 0][ct], mk);
        }
      }
      const __amdgpu_buffer_rsrc_t dst = ssm_rows(po + (int64_t)t * C * o_st, o_st, min(sg.n - t * C, C), P * S);
#pragma unroll
      for (int it = 0; it < RT; ++it) {
        const uint32_t o = (uint32_t)(16 * it + m) * (uint32_t)o_st + (uint32_t)(col0 + 4 * q) * S;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          settle(y[it][ct]);
          ssm_store4<TI>(dst, o + 16 * ct * S, y[it][ct]);
        }
      }
      // the next block's M
      form_m(smem + rb * D::bc, (const float*)(smem + D::o_w + (((t + 1) & (D::RW - 1)) * HP + hh) * D::WB),
             smem + D::o_g + (rb * HP + hh) * D::GB, smem + D::o_m + (((t + 1) & 1) * HP + hh) * D::MB);
    }

    if constexpr (OUT) {
      // read again: its registers serve the next block's M meanwhile
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int tu = 0; tu < TU; ++tu)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) xu[tu][ct] = cols.column(sX, ct, tu);
    }
    // the state update
    auto update = [&](auto terms) {
      constexpr int TERMS = decltype(terms)::value;
      auto age = [&](int tu, int nt) {  // before the tile's first product
        if (tu > 0) return;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e) H[nt][ct][e] *= alpha;
      };
#pragma unroll
      for (int tu = 0; tu < TU; ++tu) {
        // w = d 2^(the block's sum - the sum up to the token)
        f32x4 w0 = *(const f32x4*)(w + 16 * TPU * tu + 4 * q);
        if (tu == 0) w0 *= e1;
        if constexpr (S == 2) {
          const f32x4 w1 = *(const f32x4*)(w + 16 + 4 * q);
          bf16x8 a[TERMS][CT];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const uint4 x8 = __builtin_bit_cast(uint4, xu[tu][ct]);
            const uint32_t x2[4] = {x8.x, x8.y, x8.z, x8.w};
            uint32_t k[4][TERMS];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const f32x4& we = e < 2 ? w0 : w1;
              ssm_terms<TERMS>(__uint_as_float(x2[e] << 16) * we[2 * (e & 1)],
                               __uint_as_float(x2[e] & 0xffff0000u) * we[2 * (e & 1) + 1], k[e]);
            }
#pragma unroll
            for (int i = 0; i < TERMS; ++i)
              a[i][ct] = __builtin_bit_cast(bf16x8, make_uint4(k[0][i], k[1][i], k[2][i], k[3][i]));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const U b = rows.column(sB, nt, tu, l8 >> 3);
            age(tu, nt);
#pragma unroll
            for (int i = 0; i < TERMS; ++i)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a[i][ct]);
          }
        } else {
          f32x4 a[CT];
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int e = 0; e < 4; ++e) a[ct][e] = xu[tu][ct][e] * w0[e];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const U b = rows.column(sB, nt, tu, l8 >> 3);
            age(tu, nt);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) mma_unit<false>(H[nt][ct], b, a[ct]);
          }
        }
      }
    };
    if (!OUT || S == 4 || third) update(SsmInt<3>{});
    else update(SsmInt<2>{});
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) settle(H[nt][ct]);
  }

  __builtin_amdgcn_s_waitcnt(ssm_vmcnt(0));  // no copy may land after the workgroup's end
  if constexpr (OUT) {
    if (sg.first && sg.last && p.final_state) {  // (of longer sequences the join writes it)
      asm volatile("" : "+v"(l8));
      const int q = l8 >> 7, m = (l8 >> 3) & 15;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p.final_state[so + (int64_t)(ssm_state_row<TI, N>(nt, q) + e) * P + col0 + 16 * ct + m] = H[nt][ct][e];
    }
  } else {
    float* dst = slot + (int64_t)p.heads * state_elems;  // the next slot
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) *(f32x4*)(dst + fr + (nt * CT + ct) * 256) = H[nt][ct];
    if (wh == 0 && lane == 0) p.seg_decay[(int64_t)sg.slot * p.heads + h] = decay;
  }
}

// The segments of a packed batch: per segment a row (sequence, first token,
// length, segment), and each sequence's first segment.  Ends are clamped into
// [previous end, T], so that a malformed table can only give wrong results.
// One workgroup, a sequence per thread and round, the scans over waves by
// shuffles; each thread writes its own sequence's rows, or, of a sequence of
// many segments, all threads do.  Sequences of two or more segments are
// counted in the same scan and listed with their segments once more.  Bound by
// its two trips to memory and four barriers (4.0 to 5.5 us for 64 prompts).
//
// Up to kSsmSort segments are put in the order of their lengths.  Workgroups
// take a place in every compute unit before any takes a second one: where two
// rounds hold all segments, the longest ones go first, from the shortest of
// them up, and the rest from the longest of them down, so that the longest
// share a compute unit with the shortest (or with none); else the longest go
// first.  64 prompts of 200 to 4096 tokens x 16 heads of 64 columns: 430 -> 325
// us when it was built; 128 of them 765 -> 583.
constexpr int kSsmTableThreads = 1024;
constexpr int kSsmSort = 512;

__global__ __launch_bounds__(kSsmTableThreads) void ssm_table_kernel(SsmTable p) {
  __shared__ int s_end[16], s_cut[16], s_long[kSsmTableThreads][6], s_longs;
  __shared__ int64_t s_sum[16];
  __shared__ int4 s_row[kSsmSort];
  const bool sort = p.max_segs <= kSsmSort;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // of the rounds before: the end, the segments with the slots above them, the
  // cut sequences
  int carry_end = 0, carry_cut = 0;
  int64_t carry = 0;
  if (tid == 0) p.seg_off[0] = 0;
  for (int base = 0; base < p.n_seq; base += kSsmTableThreads) {
    const int i = base + tid;
    int64_t e64 = 0;
    if (i < p.n_seq) e64 = p.cu_i64 ? ((const int64_t*)p.cu)[i + 1] : ((const int32_t*)p.cu)[i + 1];
    int end = (int)min(max(e64, (int64_t)0), (int64_t)p.t_total);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(end, off);
      if (lane >= off) end = max(end, o);
    }
    if (lane == 63) s_end[wave] = end;
    if (tid == 0) s_longs = 0;
    __syncthreads();
    int before = carry_end;  // the largest end of the waves before
    for (int k = 0; k < wave; ++k) before = max(before, s_end[k]);
    const int prev = __shfl_up(end, 1);
    const int start = max(lane > 0 ? prev : 0, before);
    end = max(end, before);
    // (unsigned: a segment may be as long as all tokens)
    auto segments = [&](int tokens) { return (int)(((unsigned)tokens + (unsigned)p.seg_len - 1) / (unsigned)p.seg_len); };
    const int n = i < p.n_seq ? segments(end - start) : 0;
    const bool cut = n > 1;
    const int64_t own = n + ((int64_t)(cut ? n + 1 : 0) << 32);
    const uint64_t cuts = __ballot(cut);
    int64_t sum = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t o = __shfl_up(sum, off);
      if (lane >= off) sum += o;
    }
    if (lane == 63) {
      s_sum[wave] = sum;
      s_cut[wave] = __popcll(cuts);
    }
    __syncthreads();
    int64_t at = carry + sum - own;
    int nth = carry_cut + __popcll(cuts & ((1ull << lane) - 1));  // of the cut sequences
    const int waves = min((p.n_seq - base + 63) / 64, 16);  // the others add nothing
#pragma unroll 4
    for (int k = 0; k < waves; ++k) {
      carry_end = max(carry_end, s_end[k]);
      carry += s_sum[k];
      carry_cut += s_cut[k];
      if (k < wave) {
        at += s_sum[k];
        nth += s_cut[k];
      }
    }
    const int first = (int)(uint32_t)at, slot = cut ? (int)(at >> 32) : -1;
    if (i < p.n_seq) p.seg_off[i + 1] = first + n;
    if (cut && p.cuts && nth < p.max_cuts) *(int4*)(p.cuts + 4 * ((int64_t)nth + 1)) = make_int4(i, slot, n, 0);
    // segment k of a sequence: its row, and that of a cut one once more
    auto row = [&](int seg, int seq, int from, int to, int k, int slot, int row0) {
      if (seg >= p.max_segs) return;
      const int t0 = from + k * p.seg_len, n = min(p.seg_len, to - t0);
      const int4 r = make_int4(seq, t0, n, slot < 0 ? -1 : 4 * (slot + k) + (k == 0 ? 1 : 0) + (t0 + n == to ? 2 : 0));
      if (sort) s_row[seg] = r;
      else *(int4*)(p.table + 4 * (int64_t)seg) = r;
      if (slot >= 0 && p.cuts && row0 + k < p.max_cut_segs) *(int4*)(p.cut_table + 4 * (int64_t)(row0 + k)) = r;
    };
    if (n <= 4) {
      for (int k = 0; k < n; ++k) row(first + k, i, start, end, k, slot, slot - nth);
    } else {
      const int l = atomicAdd(&s_longs, 1);  // (the order does not matter)
      s_long[l][0] = first;
      s_long[l][1] = i;
      s_long[l][2] = start;
      s_long[l][3] = end;
      s_long[l][4] = slot;
      s_long[l][5] = slot - nth;
    }
    __syncthreads();
    for (int l = 0; l < s_longs; ++l) {
      const int from = s_long[l][2], to = s_long[l][3];
      for (int k = tid; k < segments(to - from); k += kSsmTableThreads)
        row(s_long[l][0] + k, s_long[l][1], from, to, k, s_long[l][4], s_long[l][5]);
    }
    __syncthreads();
  }
  if (tid == 0 && p.cuts) {
    // (a cut sequence has one slot more than segments)
    *(int4*)p.cuts = make_int4(min(carry_cut, p.max_cuts), min((int)(carry >> 32) - carry_cut, p.max_cut_segs), 0, 0);
  }
  if (!sort) return;
  const int total = min((int)(uint32_t)carry, p.max_segs);
  if (tid >= total) return;
  const int4 own = s_row[tid];
  int rank = 0;
  for (int k = 0; k < total; ++k) {
    const int n = s_row[k].z;
    rank += n > own.z || (n == own.z && k < tid);
  }
  if (total > p.round && total <= 2 * p.round && rank < p.round) rank = p.round - 1 - rank;
  *(int4*)(p.table + 4 * (int64_t)rank) = own;
}

hipError_t launch_ssm_table(const SsmTable& p, hipStream_t s) {
  hipLaunchKernelGGL(ssm_table_kernel, dim3(1), dim3(kSsmTableThreads), 0, s, p);
  return hipGetLastError();
}

// Joins a sequence's segments: the state before segment s is its
// predecessor's end state plus the predecessor's decay times the state before
// that one; after the last, the final state.  A thread takes four elements of
// a (sequence, head) state; `parts` workgroups share the vecs of one.  The
// order is a chain, so eight slots are asked for at once: bound by that trip
// to memory (16 heads x 16 segments 6.8 us, 48 heads x 10 segments 9.9 us).
constexpr int kSsmJoinThreads = 256;

template <typename TI, int N, int P>
__global__ __launch_bounds__(kSsmJoinThreads) void ssm_join_kernel(SsmParams p, int parts) {
  constexpr int VECS = N * P / 4, NT = N / 16;
  const int unit = blockIdx.x / parts, part = blockIdx.x - unit * parts;
  const int nth = unit / p.heads, h = unit - nth * p.heads;  // of the cut sequences
  int seq = nth, s0 = seq * (p.segs_per_seq + 1), s1 = s0 + p.segs_per_seq;  // (s1: the end state's)
  if (p.packed) {
    const int4 row = *(const int4*)(p.cuts + 4 * ((int64_t)nth + 1));
    if (nth >= p.cuts[0]) return;
    seq = row.x;
    s0 = row.y;
    s1 = s0 + row.z;
  }
  const int64_t step = (int64_t)p.heads * VECS;
  for (int at = part * kSsmJoinThreads + threadIdx.x; at < VECS; at += parts * kSsmJoinThreads) {
    f32x4* v = (f32x4*)p.slots + ((int64_t)(s0 + 1) * p.heads + h) * VECS + at;
    const float* dec = p.seg_decay + (int64_t)(s0 + 1) * p.heads + h;
    f32x4 end = zero4();
    if (p.final_state) end = v[(s1 - (s0 + 1)) * step];
    const float last = dec[(int64_t)(s1 - s0 - 2) * p.heads];
    f32x4 carry = *v;
    // a batch of slots is asked for at once (past the last one it is read again)
    constexpr int BATCH = 8;
    for (int s = s0 + 2; s < s1; s += BATCH) {
      f32x4 e[BATCH];
      float d[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int k = min(s + i, s1 - 1) - (s0 + 1);
        e[i] = v[k * step];
        d[i] = dec[(int64_t)(k - 1) * p.heads];
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (s + i >= s1) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) carry[j] = e[i][j] + d[i] * carry[j];
        v[(s + i - (s0 + 1)) * step] = carry;
      }
    }
    if (p.final_state) {
      // the fragment's place in the state (see ssm_kernel): wave's columns, tile, lane
      const int lane = at & 63, nt = (at >> 6) % NT, wave = (at >> 6) / NT;
      float* dst = p.final_state + (((int64_t)seq * p.heads + h) * N + ssm_state_row<TI, N>(nt, lane >> 4)) * P + 16 * wave + (lane & 15);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[j * P] = end[j] + last * carry[j];
    }
  }
}

// ---------------------------------------------------------------------------
// One token per sequence: reads and writes the state once, so it is bound by
// HBM.  A workgroup takes CB columns of one head's state; each thread holds
// four adjacent columns of a band of rows, read and written with 16-byte
// accesses; the contraction with c is reduced over the bands through LDS.
// All of a thread's rows are asked for before the first is used, and the
// state, which nothing reads before the next token, goes past the caches
// (nontemporal: 256 sequences x 16 heads of 128 x 128 in 96 -> 90 us, 6.0 TB/s
// where a large copy reaches 4.8; 16 sequences 10.7 -> 8.2 us).  A workgroup
// takes 16 KiB of state, N by 4096 / N columns: at 512 x 16 heads of 64 x 128
// 92 us in 64 columns, 108 in 32, 99 in 128; of 32 x 128 46 us in 128 and 88
// in 32; of 128 x 128 (256 sequences) 93 us in 32, 98 in 64.  One sequence x
// 48 heads: 3.8 us, the launch and two trips.

template <int N, int P>
struct SsmStepShape {
  static constexpr int CB = P < 4096 / N ? P : 4096 / N;  // columns per workgroup
  static constexpr int CG = CB / 4;                       // column groups
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
  for (int r = 0; r < RPT; ++r) hreg[r] = __builtin_nontemporal_load((const f32x4*)(Hs + r * P));
  const TI* br = (const TI*)p.b + (int64_t)i * p.b_st + (int64_t)grp * p.b_sh + r0;
  const TI* cr = (const TI*)p.c + (int64_t)i * p.c_st + (int64_t)grp * p.c_sh + r0;
  const f32x4 x = load4<TI>((const TI*)p.x + (int64_t)i * p.x_st + (int64_t)h * p.x_sh + c0);
  const float d = ssm_step_size(p.dt_bias ? p.dt_bias[h] : 0.f, p.dt[(int64_t)i * p.dt_st + (int64_t)h * p.dt_sh],
                                p.softplus);
  const float a = expf(ssm_rate(p.a_log, h, 1.f) * d);
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
    __builtin_nontemporal_store(hn, (f32x4*)(Hs + r * P));
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

// Two workgroups for each compute unit, what LDS and registers hold of eight
// waves with N = 128 (one with f32 inputs and P = 128).  Where more or fewer
// would fit the same number serves: 16384 tokens x 16 heads in segments for
// 256, 512 (the choice) and 1024 workgroups take, in us, bf16 128 x 128 117,
// 115, 138; 128 x 64 in odd groups 95, 78, 95, in even ones 77, 78, 101; 128 x
// 32 105, 72, 87; 128 x 16 125, 79, 89; 16 x 128 72, 67, 73; 16 x 16 84, 55, 50
// (54 for 2048); f32 64 x 32 152, 97, 111; f32 128 x 128 297, 316, 353.
int ssm_target_groups() { return 512; }
// Two heads of 64 columns fill a workgroup of eight waves.
int ssm_group_heads(bool bf16, int p, int group) { return bf16 && p == 64 && group % 2 == 0 ? 2 : 1; }

template <typename TI, int N, int P, int HP>
static hipError_t launch_ssm_kernel(bool out, const SsmParams& p, hipStream_t s) {
  const int64_t units = (int64_t)p.max_segs * (p.heads / p.unit);
  const int64_t blocks = (units + 7) / 8 * 8 * (p.unit / HP);
  if (blocks > kLaunchThreads / (SsmShape<TI, N, P, HP, true>::THREADS)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), threads(SsmShape<TI, N, P, HP, true>::THREADS);
  if (out)
    hipLaunchKernelGGL((ssm_kernel<TI, N, P, HP, true>), grid, threads, 0, s, p);
  else
    hipLaunchKernelGGL((ssm_kernel<TI, N, P, HP, false>), grid, threads, 0, s, p);
  return hipGetLastError();
}

template <typename TI, int N, int P>
static hipError_t launch_ssm_np(bool out, const SsmParams& given, hipStream_t s) {
  SsmParams p = given;
  if (!out && p.packed) p.max_segs = p.max_cut_segs;
  // heads that go to one XCD together: those of a group, unless that leaves
  // XCDs without work
  p.unit = (int64_t)p.max_segs * (p.heads / p.group) >= 64 ? p.group : 1;
  hipError_t e;
  constexpr int HP = sizeof(TI) == 2 && P == 64 ? 2 : 1;
  if (HP > 1 && ssm_group_heads(sizeof(TI) == 2, P, p.group) == HP) {
    p.unit = std::max(p.unit, HP);
    e = launch_ssm_kernel<TI, N, P, HP>(out, p, s);
  } else {
    e = launch_ssm_kernel<TI, N, P, 1>(out, p, s);
  }
  if (out || e != hipSuccess) return e;
  // workgroups for every vector; where that is many, most of them past the
  // last cut sequence of a packed batch, fewer that go round
  const int64_t units = (int64_t)p.max_cuts * p.heads;
  const int all = (N * P / 4 + kSsmJoinThreads - 1) / kSsmJoinThreads;
  const int parts = (int)std::max<int64_t>(1, std::min<int64_t>(all, 1024 / units));
  if (units * parts > kLaunchThreads / kSsmJoinThreads) return hipErrorInvalidValue;
  hipLaunchKernelGGL((ssm_join_kernel<TI, N, P>), dim3((unsigned)(units * parts)), dim3(kSsmJoinThreads), 0, s, p,
                     parts);
  return hipGetLastError();
}

template <typename TI, int N, int P>
static hipError_t launch_ssm_step_np(const SsmStepParams& all, hipStream_t s) {
  using D = SsmStepShape<N, P>;
  const int64_t each = (int64_t)all.heads * (P / D::CB);  // workgroups of a sequence
  const int64_t most = kLaunchThreads / D::NT / each;  // sequences of a launch
  if (most < 1) return hipErrorInvalidValue;
  for (int64_t i = 0; i < all.n; i += most) {
    SsmStepParams p = all;
    p.n = (int)std::min<int64_t>(most, all.n - i);
    p.x = (const TI*)all.x + i * all.x_st;
    p.dt = all.dt + i * all.dt_st;
    p.b = (const TI*)all.b + i * all.b_st;
    p.c = (const TI*)all.c + i * all.c_st;
    p.state = all.state + i * all.heads * N * P;
    p.out = (TI*)all.out + i * all.o_st;
    hipLaunchKernelGGL((ssm_step_kernel<TI, N, P>), dim3((unsigned)(p.n * each)), dim3(D::NT), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
