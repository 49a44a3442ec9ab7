// Attention of prompts and of single tokens over a paged key-value cache on
// gfx950: out = softmax(scale q.k) v over the keys that a query sees, those
// at or before its place and, with a window, inside it or among the first
// `sinks`.
//
// Both run over tiles of keys with the running maximum m and sum l of a
// row's softmax: s = scale log2(e) q.k, m' = max(m, s), l <- 2^(m - m') l +
// sum 2^(s - m'), O <- 2^(m - m') O + sum 2^(s - m') v, out = O / l.  The
// products are formed transposed, S^T = K Q^T and O^T = V^T P^T: a query is
// then a lane's column in both, so that m, l and the rescaling are one
// value a lane, and S^T's accumulators, whose rows are keys, are P^T's
// operand as they stand.  V^T's operand comes from LDS by transposed reads.
//
// Keys and values are copied straight to LDS, row by row from wherever their
// page lies.  Rows that no query of the tile sees (behind the sequence's end,
// outside the window, in a page that is not there) are copied from a zero, so
// that whatever the cache holds there reaches no product.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdn_attn.h"
#include "gdn_tiles.h"

namespace gdn {

namespace {

__device__ const uint32_t attn_zeros[4] = {0u, 0u, 0u, 0u};

__device__ __forceinline__ int attn_quotient(const Divide& d, int n) {
  return (int)((__umulhi(d.mul, (uint32_t)n) + (uint32_t)n) >> d.shift);
}

__device__ __forceinline__ int attn_cu(const AttnParams& p, int64_t i) {
  const int64_t v = p.cu_i64 ? ((const int64_t*)p.cu)[i] : (int64_t)((const int32_t*)p.cu)[i];
  return (int)min(max(v, (int64_t)0), (int64_t)p.t_total);
}

// A length that is the same for all lanes, through the scalar cache (nothing
// writes the lengths meanwhile), so that the copies under way are not waited
// for.
__device__ __forceinline__ int attn_len(const AttnParams& p, int seq) {
  typedef const __attribute__((address_space(4))) int32_t* constant;
  const int v = ((constant)(uintptr_t)p.lens)[seq];
  return min(max(v, 0), p.max_len);
}

// Copies of 16 or 4 bytes a lane into LDS, each lane's from its own address,
// in the order of the lanes from `lds` on.  Written as assembly so that the
// compiler does not wait for them at every LDS read: the wave counts them and
// waits itself.
__device__ __forceinline__ void attn_copy16(uint32_t lds, const void* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"((uint64_t)(uintptr_t)from)
               : "memory", "m0");
}
__device__ __forceinline__ void attn_copy4(uint32_t lds, const void* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 1\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"((uint64_t)(uintptr_t)from)
               : "memory", "m0");
}

// A value that is the same for all lanes, as a scalar.
__device__ __forceinline__ uint64_t attn_scalar(uint64_t v) {
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}

// The same from a common address and a lane's offset to it.  The address may
// come out of a lane (v_readlane), and an access may read such a scalar five
// wait states later at the earliest: the compiler does not count them into
// assembly, which therefore has them itself (here and in the next one).
__device__ __forceinline__ void attn_copy16(uint32_t lds, const void* base, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(attn_scalar((uint64_t)(uintptr_t)base))
               : "memory", "m0");
}

// The same, or nothing.
__device__ __forceinline__ void attn_copy16_if(bool go, uint32_t lds, const void* base, uint32_t offset) {
  asm volatile("s_cmp_eq_u32 %3, 0\n\ts_cbranch_scc1 .Lnot%=\n\ts_mov_b32 m0, %0\n\ts_nop 1\n\t"
               "global_load_lds_dwordx4 %1, %2\n.Lnot%=:"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(attn_scalar((uint64_t)(uintptr_t)base)),
                 "s"(__builtin_amdgcn_readfirstlane((int)go))
               : "memory", "m0", "scc");
}

__device__ __forceinline__ uint32_t attn_lds(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// Waits until at most n copies (and other global accesses) are under way.
template <int N>
__device__ __forceinline__ void attn_wait() {
  static_assert(N <= 63, "more than the wave counts");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(ssm_vmcnt(N));
  asm volatile("" ::: "memory");
}
// Waits for this wave's LDS reads.
__device__ __forceinline__ void attn_wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
  asm volatile("" ::: "memory");
}

// Granule g of row r of a tile sits at granule g ^ attn_swz(r), so that the
// lanes that LDS serves together meet distinct banks: 16 rows of one granule
// (keys as an operand), and four or eight rows of 64 or 32 bytes (values by
// columns).  Rows of 128 bytes alternate between the halves of the banks.
template <int GR>
__device__ __forceinline__ int attn_swz(int r) {
  const int low = ((r >> 1) & 2) | ((r >> 3) & 1);
  return GR == 8 ? ((r & 2) << 1) | low : ((r & 3) << 2) | low;
}

// Columns of values: column 16 i + l % 16 over 16 or 32 keys (see ssm_tr).
template <typename TI, int D>
struct AttnCols {
  static constexpr int RB = D * (int)sizeof(TI), GR = RB / 16;
  uint32_t at[4];  // bf16: [0]; f32: one for each of four rows
  __device__ __forceinline__ AttnCols(int lane) {
    const int q = lane >> 4, j = lane & 15;
    if constexpr (sizeof(TI) == 2) {
      const int c = 4 * (j & 3), r = 4 * q + (j >> 2);
      at[0] = r * RB + (((c >> 3) ^ attn_swz<GR>(r)) * 16) + (c & 4) * 2;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 4 * q + e;
        at[e] = r * RB + (((j >> 2) ^ attn_swz<GR>(r)) * 16) + (j & 3) * 4;
      }
    }
  }
  __device__ __forceinline__ typename Unit<TI>::type column(const char* tile, int i, int t) const {
    if constexpr (sizeof(TI) == 2) {
      const char* a = tile + (at[0] ^ (i * 32)) + t * 32 * RB;
      return ssm_tr(a, a + 16 * RB);
    } else {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const float*)(tile + (at[e] ^ (i * 64)) + t * 16 * RB);
      return v;
    }
  }
};

// ---------------------------------------------------------------------------
// 16 queries of a wave against tiles of 16 TT keys

template <typename TI, int D, int TT>
struct AttnCore {
  static constexpr int S = sizeof(TI), RB = D * S, GR = RB / 16;
  static constexpr int NU = RB / 64;  // operand units along d
  static constexpr int NC = D / 16;   // column tiles of O
  using U = typename Unit<TI>::type;
  U q[NU];
  f32x4 o[NC];  // O^T: d 16 i + 4 (l / 16) + e, query l % 16
  float m, l;   // l: this lane's keys alone

  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] = zero4();
  }
  // the queries' rows, or zeros
  static __device__ __forceinline__ void load(U (&q)[NU], const char* row, bool live, int lane) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (live) v = ld16(row + (4 * u + (lane >> 4)) * 16);
      q[u] = __builtin_bit_cast(U, v);
    }
  }
  // s[t][e]: key 16 t + 4 (l / 16) + e, query l % 16
  __device__ __forceinline__ void scores(const char* k, f32x4 (&s)[TT], int lane) const {
    const int r = lane & 15, g = lane >> 4;
    const uint32_t at = r * RB + ((g ^ attn_swz<GR>(r)) * 16);
#pragma unroll
    for (int t = 0; t < TT; ++t) s[t] = zero4();
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const U a = *(const U*)(k + (at ^ (u * 64)) + t * 16 * RB);
        mma_unit<false>(s[t], a, q[u]);
      }
#pragma unroll
    for (int t = 0; t < TT; ++t) settle(s[t]);
  }
  // a - b with both as they are: a score's product with the scale joined to it
  // would leave the largest one's rounding as an exponent.
  static __device__ __forceinline__ float minus(float a, float b) {
#pragma clang fp contract(off)
    return a - b;
  }
  // Takes a tile of scores in: s becomes the weights.
  __device__ __forceinline__ void weigh(f32x4 (&s)[TT]) {
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, s[t][e]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    top = fmaxf(m, top);
    // (a row that has seen nothing yet: weights of 2^-inf)
    const float from = top == -INFINITY ? 0.f : top;
    const float keep = __builtin_amdgcn_exp2f(m - from);
    m = top;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[t][e] = __builtin_amdgcn_exp2f(minus(s[t][e], from));
        sum += s[t][e];
      }
    l = l * keep + sum;
    if (__any(keep != 1.f)) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= keep;
    }
  }
  // O^T += V^T P^T; bf16 weights as two terms, hi and what it leaves, which
  // cost nothing where memory is waited for: within 2^-16 of the weight.
  __device__ __forceinline__ void add(const char* v, const f32x4 (&s)[TT], int lane) {
    const AttnCols<TI, D> cols(lane);
    if constexpr (S == 2) {
      static_assert(TT == 2, "two key tiles an operand unit");
      bf16x8 hi, lo;
      ssm_split2<false>(s[0], s[1], hi, lo);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const bf16x8 a = cols.column(v, i, 0);
        mma_unit<false>(o[i], a, hi);
        mma_unit<false>(o[i], a, lo);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) mma_unit<false>(o[i], cols.column(v, i, t), s[t]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) settle(o[i]);
  }
  // the whole sum of the row's weights
  __device__ __forceinline__ float total() const {
    float a = l;
    a += __shfl_xor(a, 16);
    a += __shfl_xor(a, 32);
    return a;
  }
  __device__ __forceinline__ void store(char* row, int lane) const {
    const float sum = total(), inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    if (!row) return;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      store4<TI>((TI*)row + 16 * i + 4 * (lane >> 4), o[i][0] * inv, o[i][1] * inv, o[i][2] * inv, o[i][3] * inv);
  }
};

// ---------------------------------------------------------------------------
// single tokens
//
// The queries of a key head's group (16 at most at a time) are a tile's
// columns, and memory is all that counts: every key and value once.  All
// tiles of all (sequence, key head) pairs are one list, cut in equal parts
// over the waves, so that ragged lengths, one long sequence or many short ones
// load the chip alike.  A wave works by itself, without barriers: its ring in
// LDS holds two tiles of keys and of values, the next under way while one is
// used, and the table's entries of the one after.  A wave whose part ends
// inside a pair leaves m, l and O to the join.

template <typename TI, int D>
struct StepShape {
  static constexpr int TT = sizeof(TI) == 2 ? 2 : 1, TW = 16 * TT;  // keys of a tile
  static constexpr int RB = D * (int)sizeof(TI), GR = RB / 16, TILE = TW * RB;
  static constexpr int NW = 131072 / (4 * TILE);  // waves of a workgroup
  static constexpr int PIECES = TW * GR / 64;     // copies of a tile
  static constexpr int ring = 4 * TILE, entries = NW * ring, total = entries + NW * 2 * 256;
  static_assert(total <= 163840 && NW >= 1 && NW <= 16, "LDS");
};

// A tile of the list: its pair, its number among the pair's, and what that
// pair's query sees: the tiles of the sinks, then those from `from` on.
struct StepTile {
  int seq, unit, kh, tile, tiles;
  int len, low, from, sink_tiles;  // low: the last key before the window
  __device__ __forceinline__ int first() const { return tile < sink_tiles ? tile : from + tile - sink_tiles; }
};

struct StepWork {
  const AttnParams& p;
  int units, blocks, keys;
  __device__ __forceinline__ int from(int len) const { return p.window > 0 ? max(0, len - p.window) / keys : 0; }
  __device__ __forceinline__ int sinks(int len) const {
    return p.window > 0 ? min((min(p.sinks, len) + keys - 1) / keys, from(len)) : 0;
  }
  __device__ __forceinline__ int tiles(int len) const {
    return sinks(len) + len / keys + (len % keys ? 1 : 0) - from(len);
  }
  __device__ __forceinline__ int lane_len(int64_t i) const {
    return min(max(p.lens[min(i, (int64_t)p.n_seq - 1)], 0), i < p.n_seq ? p.max_len : 0);
  }
  __device__ __forceinline__ void turn(StepTile& x, int unit) const {
    x.unit = unit;
    x.kh = blocks == 1 ? unit : unit / blocks;
  }
  __device__ __forceinline__ void enter(StepTile& x, int seq, int len) const {
    x.seq = seq;
    x.len = len;
    x.low = p.window > 0 ? len - 1 - p.window : -1;
    x.from = from(len);
    x.sink_tiles = sinks(len);
    x.tiles = tiles(len);
  }
  // The next tile of the list (there is one).
  __device__ __forceinline__ void next(StepTile& x, int lane) const {
    if (++x.tile < x.tiles) return;
    x.tile = 0;
    if (x.unit + 1 < units) {
      turn(x, x.unit + 1);
      return;
    }
    turn(x, 0);
    int seq = x.seq + 1;
    if (attn_len(p, seq) == 0) {  // empty ones, 64 at a time
      uint64_t some;
      while ((some = __ballot(lane_len((int64_t)seq + lane) > 0)) == 0) seq += 64;
      seq += __ffsll((unsigned long long)some) - 1;
    }
    seq = __builtin_amdgcn_readfirstlane(seq);
    enter(x, seq, attn_len(p, seq));
  }
};

__device__ __forceinline__ int64_t wave_upto(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int64_t wave_pick(int64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

template <typename TI, int D>
__global__ __launch_bounds__((64 * StepShape<TI, D>::NW)) void step_kernel(AttnParams p) {
  using H = StepShape<TI, D>;
  using Core = AttnCore<TI, D, H::TT>;
  constexpr int TT = H::TT, TW = H::TW, GR = H::GR, P = H::PIECES, PR = 64 / GR;
  __shared__ __attribute__((aligned(1024))) char smem[H::total];
  const int lane = threadIdx.x & 63;
  const int in_group = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wave = blockIdx.x * H::NW + in_group;
  char* ring = smem + in_group * H::ring;                 // two stages of keys, then values
  const int* entries = (const int*)(smem + H::entries + in_group * 512);
  const uint32_t ring_at = attn_lds(ring), entries_at = attn_lds(entries);

  StepWork w{p, 0, (p.group + kDecodeHeads - 1) / kDecodeHeads, TW};
  w.units = p.kv * w.blocks;

  // the wave's part [a, b) of the list: lane l sums the tiles of the sequences
  // [l c, (l + 1) c), c a 64th of all
  const int64_t c = ((int64_t)p.n_seq + 63) / 64;
  int64_t sum = 0;
  int mine_len = 0;  // (the lane's only one's)
  for (int64_t i = lane * c; i < (lane + 1) * c; i += 8) {
    int len[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) len[k] = w.lane_len(i + k);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += i + k < (lane + 1) * c ? w.tiles(len[k]) : 0;
    mine_len = len[0];
  }
  const int64_t upto = wave_upto(sum, lane);
  const int64_t all = wave_pick(upto, 63) * w.units;
  const int64_t each = all >> p.waves_log2, more = all - (each << p.waves_log2);
  const int64_t a = wave * each + min((int64_t)wave, more), b = a + each + (wave < more ? 1 : 0);
  int chain = 0, chain_seq = 0, chain_unit = 0;

  if (a < b) {
    StepTile x;
    int64_t first;  // of the pair's tiles
    {
      const uint64_t past = __ballot(upto * w.units > a);
      const int at = __ffsll((unsigned long long)past) - 1;
      int64_t before = wave_pick(upto - sum, at);
      int64_t i0 = at * c;
      if (c > 1) {  // the sequence among the lane's, 64 at a time
        int64_t mine, inner;
        uint64_t hit;
        for (;;) {
          mine = i0 + lane < (at + 1) * c ? w.tiles(w.lane_len(i0 + lane)) : 0;
          inner = wave_upto(mine, lane);
          hit = __ballot((before + inner) * w.units > a);
          if (hit) break;
          before += wave_pick(inner, 63);
          i0 += 64;
        }
        const int k = __ffsll((unsigned long long)hit) - 1;
        before += wave_pick(inner - mine, k);
        i0 += k;
      }
      const int seq = __builtin_amdgcn_readfirstlane((int)i0);
      w.enter(x, seq, c > 1 ? attn_len(p, seq) : __builtin_amdgcn_readlane(mine_len, at));
      const int64_t rest = a - before * w.units;
      const int unit = rest >> 31 ? (int)(rest / x.tiles) : (int)((uint32_t)rest / (uint32_t)x.tiles);
      w.turn(x, __builtin_amdgcn_readfirstlane(unit));
      x.tile = __builtin_amdgcn_readfirstlane((int)(rest - (int64_t)unit * x.tiles));
      first = a - x.tile;
    }

    const auto live = [&](const StepTile& t, int j) { return j < t.len && (j > t.low || j < p.sinks); };
    // The table's entries of a tile, one a lane, into one of two rows.
    const auto ask = [&](const StepTile& t, bool go, int row) {
      const int j = t.first() * TW + lane;
      const void* from = p.lens;
      if (go && lane < TW && live(t, j)) from = p.table + t.seq * p.table_st + attn_quotient(p.page, j);
      attn_copy4(entries_at + row * 256, from);
    };
    // The keys, then the values of a tile whose entries have come; which of
    // its keys there are.  Where all are and pages keep a piece's PR rows
    // together, a piece's address is its first row's and lanes' offsets to
    // it; else each lane has an address of its own.
    const bool even = p.page.d % PR == 0;
    const uint32_t g0 = ((lane % GR) ^ attn_swz<GR>(lane / GR)) * 16;
    const uint32_t k_row = lane / GR * (uint32_t)p.k_st, v_row = lane / GR * (uint32_t)p.v_st;
    const auto fetch = [&](const StepTile& t, bool go, int row, int stage) -> uint32_t {
      const int j = t.first() * TW + lane;
      const int in = j - attn_quotient(p.page, j) * (int)p.page.d;
      const int page = entries[row * 64 + (lane & (TW - 1))];
      const uint32_t there =
          (uint32_t)__ballot(go && lane < TW && live(t, j) && (uint32_t)page < (uint32_t)p.pages);
      const uint64_t ka = (uint64_t)(uintptr_t)p.k + t.kh * p.k_sh + page * p.k_sp + in * p.k_st;
      const uint64_t va = (uint64_t)(uintptr_t)p.v + t.kh * p.v_sh + page * p.v_sp + in * p.v_st;
      const uint32_t to = ring_at + 2 * stage * H::TILE;
      if (even && there == (TW == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
        for (int kind = 0; kind < 2; ++kind)
#pragma unroll
          for (int i = 0; i < P; ++i)
            attn_copy16(to + kind * H::TILE + i * 1024, (const void*)(uintptr_t)wave_pick(kind ? va : ka, i * PR),
                        (g0 ^ (attn_swz<GR>(i * PR) * 16)) + (kind ? v_row : k_row));
      } else {
#pragma unroll
        for (int kind = 0; kind < 2; ++kind)
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int r = i * PR + lane / GR;
            const uint64_t from = __shfl(kind ? va : ka, r) + (g0 ^ (attn_swz<GR>(i * PR) * 16));
            attn_copy16(to + kind * H::TILE + i * 1024, (there >> r) & 1u ? (const void*)(uintptr_t)from : attn_zeros);
          }
      }
      return there;
    };
    Core core;
    typename Core::U q[Core::NU];  // of the next tile's pair
    const int r = lane & 15;
    const auto head = [&](const StepTile& t) { return t.kh * p.group + (t.unit - t.kh * w.blocks) * kDecodeHeads; };
    const auto heads = [&](const StepTile& t) { return min(kDecodeHeads, (t.kh + 1) * p.group - head(t)); };
    const auto query = [&](const StepTile& t) {
      core.load(q, (const char*)p.q + t.seq * p.q_st + (head(t) + r) * p.q_sh, r < heads(t), lane);
    };

    StepTile now = x, then = x;
    uint32_t there, there_then = 0;
    ask(x, true, 0);
    query(x);
    attn_wait<0>();
    there = fetch(now, true, 0, 0);
    if (a + 1 < b) w.next(x, lane);
    then = x;
    ask(x, a + 1 < b, 1);
    bool fresh = true;
    for (int64_t t = a; t < b; ++t) {
      const int stage = (int)(t - a) & 1;
      attn_wait<0>();  // this tile, the next one's entries, a new pair's queries
      attn_wait_lds();
      if (fresh) {
        core.reset();
#pragma unroll
        for (int u = 0; u < Core::NU; ++u) core.q[u] = q[u];
        fresh = false;
      }
      // entries of the tile after the next
      if (t + 2 < b) w.next(x, lane);
      ask(x, t + 2 < b, stage);
      if (now.tile + 1 == now.tiles && t + 1 < b) query(then);
      there_then = fetch(then, t + 1 < b, stage ^ 1, stage ^ 1);
      f32x4 s[TT];
      core.scores(ring + 2 * stage * H::TILE, s, lane);
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[k][e] *= p.scale;
      if (there != (TW == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
        for (int k = 0; k < TT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[k][e] = (there >> (16 * k + 4 * (lane >> 4) + e)) & 1u ? s[k][e] : -INFINITY;
      }
      core.weigh(s);
      core.add(ring + (2 * stage + 1) * H::TILE, s, lane);
      if (now.tile + 1 == now.tiles || t + 1 == b) {
        fresh = true;
        const bool begun = first >= a;
        if (begun && now.tile + 1 == now.tiles) {
          core.store(r < heads(now) ? (char*)p.out + now.seq * p.o_st + (head(now) + r) * p.o_sh : nullptr, lane);
          if (p.by_pair && lane == 0) ((int4*)p.chains)[now.seq * w.units + now.unit] = make_int4(0, 0, 0, 0);
        } else {
          // a part: of a pair begun here the second slot
          float* part = p.parts + (2 * (int64_t)wave + (begun ? 1 : 0)) * attn_part_floats(D);
          const float sum = core.total();
          if (r < heads(now)) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) *(f32x4*)(part + r * D + 16 * i + 4 * (lane >> 4)) = core.o[i];
            if (lane < 16) {
              part[16 * D + r] = core.m;
              part[16 * D + 16 + r] = sum;
            }
          }
          if (begun) {
            // the wave of the pair's last tile
            const int64_t end = first + now.tiles - 1;
            const int64_t last = end < more * (each + 1) ? end / (each + 1) : more + (end - more * (each + 1)) / each;
            chain = (int)(last - wave) + 1;
            chain_seq = now.seq;
            chain_unit = now.unit;
            if (p.by_pair && lane == 0)
              ((int4*)p.chains)[now.seq * w.units + now.unit] = make_int4(chain, chain_seq, chain_unit, wave);
          }
        }
        first += now.tiles;
      }
      now = then;
      then = x;
      there = there_then;
    }
    attn_wait<0>();  // no copy may land after the workgroup's end
  }
  if (!p.by_pair && lane == 0) ((int4*)p.chains)[wave] = make_int4(chain, chain_seq, chain_unit, wave);
  // sequences that hold nothing
  for (int64_t i = wave; i < p.n_seq; i += p.waves) {
    if (attn_len(p, (int)i) != 0) continue;
    for (int g = lane; g < p.heads * GR; g += 64)
      st16((char*)p.out + i * p.o_st + (g / GR) * p.o_sh + (g % GR) * 16, make_uint4(0u, 0u, 0u, 0u));
    if (p.by_pair)
      for (int u = lane; u < w.units; u += 64) ((int4*)p.chains)[i * w.units + u] = make_int4(0, 0, 0, 0);
  }
}

// Joins the parts of the chains, PER of them a workgroup of WAVES waves: a lane
// takes four elements of a head.  A chain of at most kShortChain parts is one
// wave's, a longer one all waves', each with every WAVES-th part.
constexpr int kShortChain = 32;

template <typename TI, int D, int WAVES, int PER>
__global__ __launch_bounds__((64 * WAVES)) void join_kernel(AttnParams p) {
  constexpr int W = D / 4, BATCH = 8;
  __shared__ f32x4 s_o[WAVES * 64];
  __shared__ float s_m[WAVES * 64], s_l[WAVES * 64];
  const int lane = threadIdx.x & 63, sub = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int blocks = (p.group + kDecodeHeads - 1) / kDecodeHeads;
  const int r = (blockIdx.y * 64 + lane) / W, x = lane % W;
  int4 chains[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) chains[k] = ((const int4*)p.chains)[blockIdx.x * PER + k];

  float m, l;
  f32x4 o;
  int heads, h0;
  // the parts first, first + step, .. of a chain
  const auto gather = [&](const int4& c, int first, int step) {
    const int n = c.x, kh = blocks == 1 ? c.z : c.z / blocks;
    h0 = kh * p.group + (c.z - kh * blocks) * kDecodeHeads;
    heads = min(kDecodeHeads, (kh + 1) * p.group - h0);
    const int rr = min(r, heads - 1);
    m = -INFINITY;
    l = 0.f;
    o = zero4();
    for (int i0 = first; i0 < n; i0 += step * BATCH) {
      float pm[BATCH], pl[BATCH];
      f32x4 po[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        // part 0 is the wave's second slot, the others are the next waves' first
        const int i = min(i0 + k * step, n - 1);
        const float* part = p.parts + (2 * (int64_t)(c.w + i) + (i == 0 ? 1 : 0)) * attn_part_floats(D);
        pm[k] = part[16 * D + rr];
        pl[k] = part[16 * D + 16 + rr];
        po[k] = *(const f32x4*)(part + rr * D + 4 * x);
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        pm[k] = i0 + k * step < n ? pm[k] : -INFINITY;
        pl[k] = i0 + k * step < n ? pl[k] : 0.f;
        top = fmaxf(top, pm[k]);
      }
      const float from = top == -INFINITY ? 0.f : top, keep = __builtin_amdgcn_exp2f(m - from);
      m = top;
      l *= keep;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] *= keep;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float f = __builtin_amdgcn_exp2f(pm[k] - from);
        l += f * pl[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += i0 + k * step < n ? f * po[k][e] : 0.f;
      }
    }
  };
  const auto store = [&](const int4& c) {
    if (r >= heads) return;
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    store4<TI>((TI*)((char*)p.out + c.y * p.o_st + (h0 + r) * p.o_sh) + 4 * x, o[0] * inv, o[1] * inv, o[2] * inv,
               o[3] * inv);
  };

#pragma unroll
  for (int k = 0; k < PER; ++k)
    if (k % WAVES == sub && chains[k].x > 0 && chains[k].x <= kShortChain) {
      gather(chains[k], 0, 1);
      store(chains[k]);
    }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (chains[k].x <= kShortChain) continue;
    gather(chains[k], sub, WAVES);
    s_o[threadIdx.x] = o;
    s_m[threadIdx.x] = m;
    s_l[threadIdx.x] = l;
    __syncthreads();
    if (sub == 0) {
#pragma unroll
      for (int i = 1; i < WAVES; ++i) m = fmaxf(m, s_m[i * 64 + lane]);
      const float from = m == -INFINITY ? 0.f : m;
      l = 0.f;
      o = zero4();
#pragma unroll
      for (int i = 0; i < WAVES; ++i) {
        const float f = __builtin_amdgcn_exp2f(s_m[i * 64 + lane] - from);
        l += f * s_l[i * 64 + lane];
        const f32x4 v = s_o[i * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += f * v[e];
      }
      store(chains[k]);
    }
    __syncthreads();
  }
}

// Few pairs make long chains, and each has a large workgroup; of many most are
// short (64 sequences x 8 heads with a window of 1024, some four parts each: 52
// us in all, with a large workgroup each 56).
template <typename TI, int D>
hipError_t launch_step(AttnParams p, hipStream_t s) {
  using H = StepShape<TI, D>;
  const int heads = std::min(p.group, kDecodeHeads);
  const int64_t pairs = (int64_t)p.n_seq * p.kv * ((p.group + kDecodeHeads - 1) / kDecodeHeads);
  const unsigned chunks = (unsigned)(heads * (D / 4) + 63) / 64;
  p.by_pair = pairs <= p.waves / 16;
  p.waves_log2 = __builtin_ctz(p.waves);
  hipLaunchKernelGGL((step_kernel<TI, D>), dim3(p.waves / H::NW), dim3(64 * H::NW), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (p.by_pair)
    hipLaunchKernelGGL((join_kernel<TI, D, 16, 1>), dim3((unsigned)pairs, chunks), dim3(1024), 0, s, p);
  else
    hipLaunchKernelGGL((join_kernel<TI, D, 4, 4>), dim3(p.waves / 4, chunks), dim3(256), 0, s, p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// prompts, f32: 16 queries a wave.  Either four waves share tiles of 32 keys for
// 64 queries, or (SPLIT) four waves (d = 256: two) share 16 queries, each with
// every fourth (second) tile, of 16 keys from d = 128 on.
// Bound by fp32 matrix instructions and what stands between them: 4096 tokens x 16
// heads 101 TFLOP/s with d = 128, 96 with 64 and 98 with 256 (a product of 8192^3:
// 153).

template <typename TI, int D, bool SPLIT>
struct TileShape {
  static constexpr int TT = SPLIT && D >= 128 ? 1 : 2, TK = 16 * TT, ROWS = SPLIT ? 16 : 64;
  static constexpr int RB = D * (int)sizeof(TI), GR = RB / 16, TILE = TK * RB;
  static constexpr int NW = SPLIT && D == 256 ? 2 : 4;  // (of rings that fit)
  static constexpr int SHARE = SPLIT ? 1 : NW;         // waves that copy a tile
  static constexpr int PIECES = TK * GR / 64 / SHARE;  // copies of a tile, a wave
  static constexpr int ring = 4 * TILE, entries = NW / SHARE * ring, total = entries + NW * 2 * 256;
  static constexpr int box = D * 64, join = NW * (box + 512);  // of a wave: O, m and l
  static_assert(PIECES >= 1 && total <= 163840 && (!SPLIT || join <= total), "LDS");
};

// Where a workgroup's queries lie: rows [row, row + n) of q, at the places
// from `place` on of a sequence whose keys start at row `start` (without a
// table).
struct TileRows {
  int seq, start, row, n, place;
};

// The tile `i` of a head's: of a packed batch sequence s has those from
// floor(cu[s] / rows) + s on, as many as it fills and some over.
__device__ __forceinline__ bool tile_rows(const AttnParams& p, int64_t i, int rows, TileRows& t) {
  int at;
  if (p.cu) {
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
      if ((int64_t)attn_cu(p, mid) / rows + mid <= i) lo = mid;
      else hi = mid - 1;
    }
    t.seq = lo;
    t.start = attn_cu(p, lo);
    t.n = attn_cu(p, (int64_t)lo + 1) - t.start;
    at = (int)min((i - ((int64_t)t.start / rows + lo)) * rows, (int64_t)p.t_total);
  } else {
    const int each = (p.seq_len + rows - 1) / rows;
    t.seq = (int)(i / each);
    t.start = t.seq * p.seq_len;
    t.n = p.seq_len;
    at = (int)(i - (int64_t)t.seq * each) * rows;
  }
  if (at < 0 || at >= t.n) return false;
  t.row = t.start + at;
  t.place = at;
  if (p.table) t.place += min(max(p.lens[t.seq], 0), p.max_len) - t.n;
  t.n = min(t.n - at, rows);
  // (the same for all lanes, kept as scalars)
  t.seq = __builtin_amdgcn_readfirstlane(t.seq);
  t.start = __builtin_amdgcn_readfirstlane(t.start);
  t.row = __builtin_amdgcn_readfirstlane(t.row);
  t.n = __builtin_amdgcn_readfirstlane(t.n);
  t.place = __builtin_amdgcn_readfirstlane(t.place);
  return true;
}

template <typename TI, int D, bool PAGED, bool SPLIT>
__global__ __launch_bounds__((64 * TileShape<TI, D, SPLIT>::NW)) void tile_kernel(AttnParams p, int tiles) {
  using H = TileShape<TI, D, SPLIT>;
  constexpr int TT = H::TT, TK = H::TK, GR = H::GR, P = H::PIECES, NW = H::NW;
  constexpr uint32_t ALL = TK == 32 ? 0xffffffffu : 0xffffu;
  __shared__ __attribute__((aligned(1024))) char smem[H::total];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int item = blockIdx.x / p.heads;  // (long tiles first)
  const int h = blockIdx.x - item * p.heads, kh = h / p.group;
  TileRows t;
  if (!tile_rows(p, tiles - 1 - item, H::ROWS, t)) return;
  const int lo = t.place, hi = t.place + t.n - 1;  // the queries' places
  const int skip = SPLIT ? 0 : wave * 16;          // to the wave's first query
  const int mine = skip + (lane & 15), place = lo + mine, wave_lo = lo + skip;
  AttnCore<TI, D, TT> core;
  core.reset();
  core.load(core.q, (const char*)p.q + (int64_t)(t.row + mine) * p.q_st + h * p.q_sh, mine < t.n, lane);

  // key tiles: those of the sinks, then those from the window's start on; a
  // wave's are every SHARE-th or, split, every NW-th
  const int end = hi / TK + (hi >= 0 ? 1 : 0);
  const int from = p.window > 0 ? max(0, max(lo, 0) - p.window + 1) / TK : 0;
  const int sinks = p.window > 0 ? min((min(p.sinks, hi + 1) + TK - 1) / TK, from) : 0;
  const int all = max(0, sinks + end - from);
  const int turns = SPLIT ? (all - wave + NW - 1) / NW : all;
  const auto tile_at = [&](int j) {  // `end` or more: none
    const int i = SPLIT ? j * NW + wave : j;
    return i < sinks ? i : from + i - sinks;
  };
  char* const ring = smem + (SPLIT ? wave * H::ring : 0);
  const uint32_t ring_at = attn_lds(ring), entries_at = attn_lds(smem + H::entries + wave * 512);
  const int* entries = (const int*)(smem + H::entries + wave * 512);
  const int low = p.window > 0 ? max(lo, 0) - p.window : -1;  // the last key before every window
  const auto live = [&](int j) { return j <= hi && (j > low || j < p.sinks); };
  const auto ask = [&](int k, int row) {
    if (!PAGED) return;
    const int j = k * TK + lane;
    const void* a = p.lens;
    if (k < end && lane < TK && live(j)) a = p.table + t.seq * p.table_st + attn_quotient(p.page, j);
    attn_copy4(entries_at + row * 256, a);
  };
  // (as the single tokens' copies)
  constexpr int PR = 64 / GR;
  const bool even = !PAGED || p.page.d % PR == 0;
  const uint32_t k_row = lane / GR * (uint32_t)p.k_st, v_row = lane / GR * (uint32_t)p.v_st;
  const auto fetch = [&](int k, int row, int stage) -> uint32_t {
    const int j = k * TK + lane;
    bool there = k < end && lane < TK && live(j);
    int page = 0, in = j;
    if (PAGED) {
      page = entries[row * 64 + lane % TK];
      there = there && (uint32_t)page < (uint32_t)p.pages;
      in = j - attn_quotient(p.page, j) * (int)p.page.d;
    } else {
      in += t.start;
    }
    const uint32_t mask = (uint32_t)__ballot(there);
    uint64_t ka = (uint64_t)(uintptr_t)p.k + kh * p.k_sh + in * p.k_st;
    uint64_t va = (uint64_t)(uintptr_t)p.v + kh * p.v_sh + in * p.v_st;
    if (PAGED) ka += page * p.k_sp, va += page * p.v_sp;
    const int first = SPLIT ? 0 : wave * PR;
    constexpr int STEP = H::SHARE * PR;
    const uint32_t to = ring_at + 2 * stage * H::TILE + (SPLIT ? 0 : wave * 1024);
    if (even && mask == ALL) {
#pragma unroll
      for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint32_t g = ((lane % GR) ^ attn_swz<GR>(first + i * STEP + lane / GR)) * 16;
          attn_copy16(to + kind * H::TILE + i * H::SHARE * 1024,
                      (const void*)(uintptr_t)wave_pick(kind ? va : ka, first + i * STEP), g + (kind ? v_row : k_row));
        }
    } else {
#pragma unroll
      for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int r = first + i * STEP + lane / GR;
          const uint64_t a = __shfl(kind ? va : ka, r) + ((lane % GR) ^ attn_swz<GR>(r)) * 16;
          attn_copy16(to + kind * H::TILE + i * H::SHARE * 1024, (mask >> r) & 1u ? (const void*)(uintptr_t)a : attn_zeros);
        }
    }
    return mask;
  };
  ask(tile_at(0), 0);
  attn_wait<0>();
  uint32_t there = fetch(tile_at(0), 0, 0), there_then;
  ask(tile_at(1), 1);
  for (int j = 0; j < turns; ++j) {
    const int stage = j & 1, j0 = tile_at(j) * TK;
    attn_wait_lds();
    ask(tile_at(j + 2), stage);
    attn_wait<PAGED ? 1 : 0>();
    if (!SPLIT) lds_barrier();
    there_then = fetch(tile_at(j + 1), stage ^ 1, stage ^ 1);
    f32x4 s[TT];
    core.scores(ring + 2 * stage * H::TILE, s, lane);
#pragma unroll
    for (int k = 0; k < TT; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[k][e] *= p.scale;
    if (!(there == ALL && j0 + TK - 1 <= wave_lo &&
          (p.window <= 0 || j0 > wave_lo + 15 - p.window || j0 + TK <= p.sinks))) {
#pragma unroll
      for (int k = 0; k < TT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int in = 16 * k + 4 * (lane >> 4) + e, at = j0 + in;
          const bool see = ((there >> in) & 1u) && at <= place && (p.window <= 0 || place - at < p.window || at < p.sinks);
          s[k][e] = see ? s[k][e] : -INFINITY;
        }
    }
    core.weigh(s);
    core.add(ring + (2 * stage + 1) * H::TILE, s, lane);
    there = there_then;
  }
  attn_wait<0>();  // no copy may land after the workgroup's end
  char* const out = mine < t.n ? (char*)p.out + (int64_t)(t.row + mine) * p.o_st + h * p.o_sh : nullptr;
  if constexpr (!SPLIT) {
    core.store(out, lane);
  } else {
    // The join: each wave ends up with its share of d.
    constexpr int NC = D / 16, MY = NC / NW;
    const float l = core.total();
    lds_barrier();
    f32x4* const box = (f32x4*)smem;
    float* const ml = (float*)(smem + NW * H::box);
#pragma unroll
    for (int i = 0; i < NC; ++i) box[(wave * NC + i) * 64 + lane] = core.o[i];
    ml[wave * 128 + lane] = core.m;
    ml[wave * 128 + 64 + lane] = l;
    lds_barrier();
    float m = -INFINITY, sum = 0.f, f[NW];
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, ml[w * 128 + lane]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      f[w] = __builtin_amdgcn_exp2f(ml[w * 128 + lane] - base);
      sum += f[w] * ml[w * 128 + 64 + lane];
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < MY; ++i) {
      f32x4 y = zero4();
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const f32x4 v = box[(w * NC + wave * MY + i) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += f[w] * v[e];
      }
      if (out) store4<TI>((TI*)out + 16 * (wave * MY + i) + 4 * (lane >> 4), y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    }
  }
}

// ---------------------------------------------------------------------------
// prompts, bf16: 32 queries a wave, tiles of 64 keys shared by four waves
//
// Bound by products and softmax in turns, neither of which fills its unit (4096
// tokens x 16 heads of 128: matrix cores busy 42 % of the time, the vector unit 43;
// behind a cache with d = 256 37 and 34): one prompt of 16384 tokens x 16 heads
// runs at 1117 TFLOP/s with d = 128, 948 with 64 and 1007 with 256, where a product
// of 16384^3 reaches 1387.  32 columns a wave give 32 x 32 x 16 products whose
// softmax is 16 scores a lane and 32 keys; at d <= 128 two waves a SIMD cover
// each other's softmax (a third would not fit LDS and registers).  Weights of
// one bf16 term: off by 2^-8 of themselves at most, as the output by its own rounding.
// Tiles of 64 keys, two stages, one barrier a tile; copies of the next tile go
// out between this one's products.  Tried and slower: groups of waves in turns
// by barriers, tiles of 32 keys with the next one's scores beside the softmax
// (119 us for 98), wave priorities.

typedef float f32x16 __attribute__((ext_vector_type(16)));

// GROUPS: of four waves, which take every GROUPS-th tile of keys and join.
template <int D, int GROUPS>
struct PromptShape {
  static constexpr int NW = 4, ROWS = 32 * NW, TK = 64;  // NW: waves of a group
  static constexpr int RB = D * 2, GR = RB / 16, TILE = TK * RB;
  static constexpr int P = TK * GR / 64 / NW;  // copies of a tile's keys, a wave
  static constexpr int ring = 4 * TILE, entries = GROUPS * ring, total = entries + GROUPS * NW * 2 * 256;
  // the join: of every wave half of O, and m and l
  static constexpr int box = 64 * D, join = 2 * NW * (box + 512);
  static_assert(total <= 163840 && (GROUPS == 1 || join <= total), "LDS");
};

constexpr int kPromptRows = PromptShape<64, 1>::ROWS;

// The n lowest bits.
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : ((uint64_t)1 << n) - 1;
}

// The larger of a lane's value and of the one 32 lanes away.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ void settle16(f32x16& a) { asm volatile("" : "+v"(a)); }

// A weight's exponent is s scale - m in one operation, m the rounded product of
// the largest s: off by m's rounding for all of a row alike, which the quotient
// of the sums does not see, but which leaves every exponent's range where m is
// past some 2^28.  Where a row of the wave has an m of 2^12 or more, the scores
// are rounded first, so that the largest one's exponent is 0.  (A row below that
// may have some tiles the one way and some the other: 2^-12 in the exponent, a
// 20th of its weights' own rounding.)  Rows below it pay nothing: 16384 tokens x
// 16 heads 1018 us with and without it (d = 128), 2250 and 2245 (256), 595 and 591
// (64).
constexpr float kFarScore = 0x1p12f;
// What a row's largest score has to pass for its maximum to be looked at again:
// 2^8 times the last one, whose weights lose nothing in fp32 or bf16; anything
// where it is far.
__device__ __forceinline__ float next_bar(float m) { return fabsf(m) >= kFarScore ? -INFINITY : m + 8.f; }
__device__ __forceinline__ void scale_scores(f32x16 (&s)[2], float scale) {
#pragma unroll
  for (int n = 0; n < 32; ++n) s[n >> 4][n & 15] *= scale;
  settle16(s[0]);  // (rounded here)
  settle16(s[1]);
}

template <int D, bool PAGED, int GROUPS>
__global__ __launch_bounds__(256 * GROUPS, (D == 256 ? 1 : 2)) void prompt_kernel(AttnParams p, int tiles) {
  using H = PromptShape<D, GROUPS>;
  constexpr int TK = H::TK, RB = H::RB, GR = H::GR, P = H::P, NS = D / 16, NC = D / 32;
  __shared__ __attribute__((aligned(1024))) char smem[H::total];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int group = wid >> 2, wave = wid & 3;
  const int half = lane >> 5, col = lane & 31;
  int rank = blockIdx.x / p.heads;
  const int hp = blockIdx.x - rank * p.heads;
  // Long tiles first.  Where the chip holds all of them at once, two a compute
  // unit, the second half the other way round.
  if (GROUPS == 1 && gridDim.x <= 512 && 2 * rank >= tiles) rank = (tiles + 1) / 2 + tiles - 1 - rank;
  const int h = p.heads % 8 == 0 ? (hp & 7) * (p.heads / 8) + (hp >> 3) : hp, kh = h / p.group;
  TileRows t;
  if (!tile_rows(p, tiles - 1 - rank, H::ROWS, t)) return;
  const int lo = t.place, hi = t.place + t.n - 1;
  const int mine = wave * 32 + col, place = lo + mine;
  const int wave_lo = lo + wave * 32, wave_hi = min(wave_lo + 31, hi);

  // (the largest score is the largest product: a scale's sign goes to q)
  const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
  const float scale = fabsf(p.scale);
  bf16x8 q[NS];
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (mine < t.n) v = ld16((const char*)p.q + (int64_t)(t.row + mine) * p.q_st + h * p.q_sh + (2 * u + half) * 16);
    v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
    q[u] = __builtin_bit_cast(bf16x8, v);
  }
  f32x16 o[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
  float m = -INFINITY, l = 0.f, bar = -INFINITY;

  // key tiles: those of the sinks, then those from the window's start on; a
  // group's are every GROUPS-th
  const int end = hi / TK + (hi >= 0 ? 1 : 0);
  const int from = p.window > 0 ? max(0, max(lo, 0) - p.window + 1) / TK : 0;
  const int sinks = p.window > 0 ? min((min(p.sinks, hi + 1) + TK - 1) / TK, from) : 0;
  const int turns = (max(0, sinks + end - from) + GROUPS - 1) / GROUPS;
  const auto tile_at = [&](int j) {  // the group's tile j; `end` or more: none
    const int i = GROUPS * j + group;
    return i < sinks ? i : from + i - sinks;
  };
  const char* const ring = smem + group * H::ring;
  const uint32_t ring_at = attn_lds(ring), entries_at = attn_lds(smem + H::entries + wid * 512);
  const int* entries = (const int*)(smem + H::entries + wid * 512);
  const int low = p.window > 0 ? max(lo, 0) - p.window : -1;  // the last key before every window
  const auto live = [&](int j) { return j <= hi && (j > low || j < p.sinks); };
  const auto ask = [&](int k, int row) {
    if (!PAGED) return;
    const int j = k * TK + lane;
    const void* a = p.lens;
    if (k < end && live(j)) a = p.table + t.seq * p.table_st + attn_quotient(p.page, j);
    attn_copy4(entries_at + row * 256, a);
  };
  const char* const k_base = (const char*)p.k + kh * p.k_sh;
  const char* const v_base = (const char*)p.v + kh * p.v_sh;
  // A tile that is there as a whole is copied from common addresses, one a
  // piece of PR rows (which pages of a multiple of PR keep together), and
  // lanes' offsets that stay; others row by row.
  constexpr int PR = 64 / GR;
  const bool even = !PAGED || p.page.d % PR == 0;
  constexpr int STEP = H::NW * PR;          // rows to the wave's next piece
  constexpr int KINDS = STEP % 16 ? 2 : 1;  // of swizzles among its pieces
  uint32_t k_off[KINDS], v_off[KINDS];
#pragma unroll
  for (int i = 0; i < KINDS; ++i) {
    const int r = i * STEP + wave * PR + lane / GR, row = PAGED ? lane / GR : wave * PR + lane / GR;
    const uint32_t g = ((lane % GR) ^ attn_swz<GR>(r)) * 16;
    k_off[i] = (uint32_t)row * (uint32_t)p.k_st + g;
    v_off[i] = (uint32_t)row * (uint32_t)p.v_st + g;
  }
  // Where a tile's rows lie: with pages the lane's key and value, and which keys
  // there are.
  struct Where {
    int tile;
    uint64_t there, ka, va;
  };
  const auto look = [&](int k, int row) {
    Where w{k, 0, 0, 0};
    const int j0 = k * TK, j = j0 + lane;
    if (!PAGED && j0 + TK - 1 <= hi && (j0 > low || j0 + TK <= p.sinks)) {
      w.there = ~0ull;
      return w;
    }
    bool is = k < end && live(j);
    if (PAGED) {
      const int page = entries[row * 64 + lane], in = j - attn_quotient(p.page, j) * (int)p.page.d;
      is = is && (uint32_t)page < (uint32_t)p.pages;
      w.ka = (uint64_t)(uintptr_t)k_base + page * p.k_sp + in * p.k_st;
      w.va = (uint64_t)(uintptr_t)v_base + page * p.v_sp + in * p.v_st;
    }
    w.there = __ballot(is);
    return w;
  };
  // Piece i of a tile that is there as a whole, keys first (`go` false:
  // nothing); all pieces of any tile.  Without pages a tile's pieces follow
  // each other by a stride.
  const int64_t k_step = STEP * p.k_st, v_step = STEP * p.v_st;
  const char *k_now = nullptr, *v_now = nullptr;
  const auto start = [&](const Where& w) __attribute__((always_inline)) {
    if (PAGED) return;
    k_now = k_base + (int64_t)(t.start + w.tile * TK) * p.k_st;
    v_now = v_base + (int64_t)(t.start + w.tile * TK) * p.v_st;
  };
  const auto copy = [&](const Where& w, uint32_t to, int i, bool go) __attribute__((always_inline)) {
    const bool values = i >= P;
    if (values) i -= P;
    const char* from;
    if (PAGED) {
      from = (const char*)(uintptr_t)wave_pick(values ? w.va : w.ka, i * STEP + wave * PR);
    } else if (values) {
      from = v_now;
      v_now += v_step;
    } else {
      from = k_now;
      k_now += k_step;
    }
    attn_copy16_if(go, to + i * H::NW * 1024 + (values ? H::TILE : 0), from,
                   values ? v_off[i % KINDS] : k_off[i % KINDS]);
  };
  const auto fetch = [&](const Where& w, uint32_t to) {
    uint64_t ka = w.ka, va = w.va;
    if (!PAGED) {
      ka = (uint64_t)(uintptr_t)k_base + (int64_t)(t.start + w.tile * TK + lane) * p.k_st;
      va = (uint64_t)(uintptr_t)v_base + (int64_t)(t.start + w.tile * TK + lane) * p.v_st;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int r = i * STEP + wave * PR + lane / GR;
      const uint64_t kr = __shfl(ka, r), vr = __shfl(va, r);
      const int g = ((lane % GR) ^ attn_swz<GR>(r)) * 16;
      const bool is = (w.there >> r) & 1u;
      attn_copy16(to + i * H::NW * 1024, is ? (const void*)(uintptr_t)(kr + g) : attn_zeros);
      attn_copy16(to + i * H::NW * 1024 + H::TILE, is ? (const void*)(uintptr_t)(vr + g) : attn_zeros);
    }
  };
  const auto stage_at = [&](int stage) { return ring_at + 2 * stage * H::TILE + wave * 1024; };

  // operand places: keys by rows, values by columns (two halves of 16 keys)
  const uint32_t k_at = col * RB + ((half ^ attn_swz<GR>(col)) * 16);
  const int vr = 4 * half + ((lane & 15) >> 2), vc = (lane & 16) + 4 * (lane & 3);
  const uint32_t v_at0 = vr * RB + (((vc >> 3) ^ attn_swz<GR>(vr)) * 16) + (vc & 4) * 2;
  const uint32_t v_at1 = (vr + 8) * RB + (((vc >> 3) ^ attn_swz<GR>(vr + 8)) * 16) + (vc & 4) * 2;

  if (PAGED) {
    ask(tile_at(0), 0);
    attn_wait<0>();
  }
  Where here = look(tile_at(0), 0);
  fetch(here, stage_at(0));
  ask(tile_at(1), 1);
  // Tiles that every query of the workgroup sees as a whole, the group's next
  // one there as a whole too: nothing is looked up for them.
  const int plain_from = p.window > 0 ? max(from, (hi - p.window >= 0 ? (hi - p.window) / TK + 1 : 0)) : 0;
  const int plain_to = min((max(lo, -1) + 1) / TK, (max(hi, -1) + 1) / TK - GROUPS);
  for (int j = 0; j < turns; ++j) {
    const int stage = j & 1;
    attn_wait_lds();
    ask(tile_at(j + 2), stage);
    attn_wait<PAGED ? 1 : 0>();
    lds_barrier();
    const int j0 = here.tile * TK;
    const bool plain = !PAGED && here.tile >= plain_from && here.tile < plain_to;
    Where next{here.tile + GROUPS, ~0ull, 0, 0};
    if (!plain) next = look(tile_at(j + 1), stage ^ 1);
    const bool whole = plain || (j0 + TK - 1 <= wave_lo && here.there == ~0ull &&
                                 (p.window <= 0 || j0 > wave_hi - p.window || j0 + TK <= p.sinks));
    const bool any = whole || (here.tile < end && wave_lo <= hi && j0 <= wave_hi &&
                               (p.window <= 0 || j0 + TK - 1 > max(wave_lo, 0) - p.window || j0 < p.sinks));
    const uint32_t to = stage_at(stage ^ 1);
    const bool go = any && next.there == ~0ull && even;
    start(next);
    if (!go) {
      if (next.there == ~0ull && even) {
#pragma unroll
        for (int i = 0; i < 2 * P; ++i) copy(next, to, i, true);
      } else {
        fetch(next, to);
      }
    }
    if (any) {
      const char* kt = ring + 2 * stage * H::TILE;
      const char* vt = kt + H::TILE;
      const auto key = [&](int u, int b) { return *(const bf16x8*)(kt + (k_at ^ (u * 32)) + b * 32 * RB); };
      const auto value = [&](int u, int i) {
        return ssm_tr(vt + (v_at0 ^ (i * 64)) + u * 16 * RB, vt + (v_at1 ^ (i * 64)) + u * 16 * RB);
      };
      const auto hide = [&](f32x16 (&s)[2]) __attribute__((always_inline)) {
        // the keys that the lane's query sees, a bit each
        uint64_t see = here.there & low_bits(place - j0 + 1);
        if (p.window > 0) see &= ~low_bits(place - j0 - p.window + 1) | low_bits(p.sinks - j0);
        see >>= 4 * half;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[b][e] = ((uint32_t)(see >> (32 * b)) >> (8 * (e >> 2) + (e & 3))) & 1u ? s[b][e] : -INFINITY;
      };
      if constexpr (D < 256) {
        constexpr int AHEAD = NS < 6 ? NS : 6;  // pairs of operands on their way
        f32x16 s[2];
        bf16x8 a[NS][2], first[NC], w[4];
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e >> 4][e & 15] = 0.f;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
          for (int b = 0; b < 2; ++b) a[u][b] = key(u, b);
        // the next tile's copies run between this one's products: one after the
        // other they would wait for the way into LDS
#pragma unroll
        for (int u = 0; u < NS; ++u) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[u][b], q[u], s[b], 0, 0, 0);
            if (u + AHEAD < NS) a[u + AHEAD][b] = key(u + AHEAD, b);
          }
          if (u < 2 * P) copy(next, to, u, go);
          __builtin_amdgcn_sched_barrier(0);
        }
        // (the first of V's operands, asked for early)
#pragma unroll
        for (int i = 0; i < NC; ++i) first[i] = value(0, i);
        settle16(s[0]);
        settle16(s[1]);
        if (!whole) hide(s);
        float top = s[0][0];
#pragma unroll
        for (int n = 1; n < 32; ++n) top = fmaxf(top, s[n >> 4][n & 15]);
        // O and l are rescaled only where the maximum has grown by more than 2^8
        float by = scale;
        if (__any(top * scale > bar)) {
          const float up = fmaxf(m, max_halves(top) * scale);
          const float keep = __builtin_amdgcn_exp2f(m - (up == -INFINITY ? 0.f : up));
          m = up;
          l *= keep;
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] *= keep;
          bar = next_bar(m);
          if (__any(fabsf(m) >= kFarScore && m != -INFINITY)) {
            scale_scores(s, scale);
            by = 1.f;
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 32; ++n) {
          const float x = __builtin_amdgcn_exp2f(s[n >> 4][n & 15] * by - base);
          sum[n & 1] += x;
          w[n >> 3][n & 7] = (bf16)x;
        }
        l += sum[0] + sum[1];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int i = 0; i < NC; ++i)
            o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(u == 0 ? first[i] : value(u, i), w[u], o[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < NC; ++i) settle16(o[i]);
      } else {
        // A wave alone on its SIMD: half a tile's softmax beside the products of the
        // other half's scores, the other half's beside those of the first one's
        // values (4096 tokens x 16 heads 186 us, one after the other 203; with two
        // waves a SIMD, d = 128, 100.3 and 98.1).  The products' operands are read
        // in their order, AHEAD of them on their way.
        constexpr int NK = 2 * NS, NV = 4 * NC, AHEAD = 8;
        f32x16 s[2];
        bf16x8 a[NK + NV], w[4];
        const auto read = [&](int n) __attribute__((always_inline)) {
          if (n < NK) a[n] = key(n % NS, n / NS);
          else if (n < NK + NV) a[n] = value((n - NK) / NC, (n - NK) % NC);
        };
        float top[2], sum[2], by = scale;
        const float before = m == -INFINITY ? 0.f : m;
        // The weights of the 16 scores of half b against a maximum, in steps of
        // `part`: a step forms exponents, the next one their powers, the one
        // after sums and rounds them, so that none waits for the one before.
        float y[16];
        const auto weigh = [&](int b, int step, int part, float base) __attribute__((always_inline)) {
#pragma unroll
          for (int e = step * part; e < min(16, (step + 1) * part); ++e) {
            y[e] = s[b][e] * by - base;
            if (b == 0) top[0] = e == 0 ? s[0][0] : fmaxf(top[0], s[0][e]);
          }
          if (step > 0) {
#pragma unroll
            for (int e = (step - 1) * part; e < min(16, step * part); ++e) y[e] = __builtin_amdgcn_exp2f(y[e]);
          }
          if (step > 1) {
#pragma unroll
            for (int e = (step - 2) * part; e < min(16, (step - 1) * part); ++e) {
              sum[b] = e == 0 ? y[0] : sum[b] + y[e];
              w[2 * b + (e >> 3)][e & 7] = (bf16)y[e];
            }
          }
        };
#pragma unroll
        for (int n = 0; n < 32; ++n) s[n >> 4][n & 15] = 0.f;
#pragma unroll
        for (int f = 0; f < AHEAD; ++f) read(f);
        // the scores of 32 keys, then of the other 32 beside the first ones'
        // weights; the next tile's copies between them
        constexpr int STEPS = NS - 3, PART = (16 + STEPS - 1) / STEPS;
#pragma unroll
        for (int f = 0; f < 2 * NS; ++f) {
          s[f / NS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[f], q[f % NS], s[f / NS], 0, 0, 0);
          read(f + AHEAD);
          if (f < 2 * P) copy(next, to, f, go);
          if (f > NS) weigh(0, f - NS - 1, PART, before);
          __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(sum[0]), "+v"(top[0]));  // (weighed here, not behind the branch)
        settle16(s[0]);
        settle16(s[1]);
        if (!whole) hide(s);
        top[1] = s[1][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top[1] = fmaxf(top[1], s[1][e]);
        // O and l are rescaled only where the maximum has grown by more than 2^8
        bool redo = false;  // (a flag: a branch over both would have O copied)
        if (!whole || __any(fmaxf(top[0], top[1]) * scale > bar)) {
          top[0] = s[0][0];
#pragma unroll
          for (int e = 1; e < 16; ++e) top[0] = fmaxf(top[0], s[0][e]);
          const float up = fmaxf(m, max_halves(fmaxf(top[0], top[1])) * scale);
          const float keep = __builtin_amdgcn_exp2f(m - (up == -INFINITY ? 0.f : up));
          m = up;
          l *= keep;
#pragma unroll
          for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] *= keep;
          bar = next_bar(m);
          redo = true;
        }
        if (redo) {
          if (__any(fabsf(m) >= kFarScore && m != -INFINITY)) {
            scale_scores(s, scale);
            by = 1.f;
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) weigh(0, i, 16, m == -INFINITY ? 0.f : m);
        }
        l += sum[0];
        // the first 32 keys' values beside the other ones' weights
        const float base = m == -INFINITY ? 0.f : m;
        constexpr int STEPS1 = 2 * NC - 3, PART1 = (16 + STEPS1 - 1) / STEPS1;
#pragma unroll
        for (int f = 0; f < 2 * NC; ++f) {
          const int u = f / NC, i = f % NC;
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[NK + f], w[u], o[i], 0, 0, 0);
          read(NK + f + AHEAD);
          if (f > 0) weigh(1, f - 1, PART1, base);
          __builtin_amdgcn_sched_barrier(0);
        }
        l += sum[1];
#pragma unroll
        for (int f = 0; f < 2 * NC; ++f) {
          const int u = 2 + f / NC, i = f % NC;
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[NK + 2 * NC + f], w[u], o[i], 0, 0, 0);
          read(NK + 2 * NC + f + AHEAD);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) settle16(o[i]);
      }
    }
    here = next;
  }
  attn_wait<0>();  // no copy may land after the workgroup's end
  l += __shfl_xor(l, 32);
  if constexpr (GROUPS == 1) {
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    if (mine < t.n) {
      bf16* out = (bf16*)((char*)p.out + (int64_t)(t.row + mine) * p.o_st + h * p.o_sh) + 4 * half;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          store4<bf16>(out + 32 * i + 8 * j, o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                       o[i][4 * j + 3] * inv);
    }
    return;
  } else {
    // The join: each group ends up with one half of d.
    lds_barrier();
    f32x4* const box = (f32x4*)smem + wid * (H::box / 16);
    float* const ml = (float*)(smem + 2 * H::NW * H::box) + wid * 128;
#pragma unroll
    for (int i = 0; i < NC / 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = group ? o[i][4 * j + e] : o[i + NC / 2][4 * j + e];
        box[(4 * i + j) * 64 + lane] = v;
      }
    ml[lane] = m;
    ml[64 + lane] = l;
    lds_barrier();
    const f32x4* const from_box = (const f32x4*)smem + (wid ^ 4) * (H::box / 16);
    const float* const from_ml = (const float*)(smem + 2 * H::NW * H::box) + (wid ^ 4) * 128;
    const float m2 = from_ml[lane], l2 = from_ml[64 + lane];
    const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.f : top;
    float f1 = __builtin_amdgcn_exp2f(m - base), f2 = __builtin_amdgcn_exp2f(m2 - base);
    const float all = l * f1 + l2 * f2, inv = all > 0.f || all != all ? 1.f / all : 0.f;
    f1 *= inv;
    f2 *= inv;
    if (mine < t.n) {
      bf16* out = (bf16*)((char*)p.out + (int64_t)(t.row + mine) * p.o_st + h * p.o_sh) + group * (D / 2) + 4 * half;
#pragma unroll
      for (int i = 0; i < NC / 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 v = from_box[(4 * i + j) * 64 + lane];
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = (group ? o[i + NC / 2][4 * j + e] : o[i][4 * j + e]) * f1 + v[e] * f2;
          store4<bf16>(out + 32 * i + 8 * j, y[0], y[1], y[2], y[3]);
        }
    }
  }
}

int64_t tiles_of(const AttnParams& p, int rows) {
  return p.cu ? (int64_t)p.t_total / rows + p.n_seq : (int64_t)p.n_seq * ((p.seq_len + rows - 1) / rows);
}

template <int D, int GROUPS>
hipError_t launch_prompt(const AttnParams& p, int tiles, hipStream_t s) {
  const dim3 grid((unsigned)((int64_t)tiles * p.heads)), threads(256 * GROUPS);
  if (p.table)
    hipLaunchKernelGGL((prompt_kernel<D, true, GROUPS>), grid, threads, 0, s, p, tiles);
  else
    hipLaunchKernelGGL((prompt_kernel<D, false, GROUPS>), grid, threads, 0, s, p, tiles);
  return hipGetLastError();
}

template <int D>
hipError_t launch_prompt(const AttnParams& p, hipStream_t s) {
  const int tiles = (int)tiles_of(p, kPromptRows);
  // Few workgroups: the last one's time is the whole call's, and one that is
  // alone on its compute unit leaves half of it idle.  Measured, two groups and
  // one, d = 128 (64): one prompt of 4096 tokens x 16 heads (512 workgroups) 82 and
  // 91 us (53 and 60), 2048 x 16 36 and 43 (24 and 31), 1024 x 16 21 and 24 (15 and
  // 18), 8192 x 8 145 and 170 (96 and 112); past 512, 4096 x 20 110 and 100 (70 and
  // 66), x 24 122 and 111, x 32 152 and 147.  With a window of 512, whose tiles are
  // alike, 2048 x 16 (256) 18.5 and 20 (12.6 and 14.3), 4096 x 16 (512) 36 and 30 (23
  // and 20), 8192 x 16 (1024) 69 and 55; of 128, 1024 x 16 12.8 and 11.5 (9 and 9).
  // Workgroups count as the grid does, a packed batch's spare one a sequence and
  // head too (4096 x 16 as a packed batch of one: 528), and any window as one that
  // shortens chains, also one that is longer than the prompt.
  if constexpr (D <= 128)
    if ((int64_t)tiles * p.heads <= (p.window > 0 ? 256 : 512)) return launch_prompt<D, 2>(p, tiles, s);
  return launch_prompt<D, 1>(p, tiles, s);
}

template <typename TI, int D, bool SPLIT>
hipError_t launch_tiles(const AttnParams& p, hipStream_t s) {
  using H = TileShape<TI, D, SPLIT>;
  const int tiles = (int)tiles_of(p, H::ROWS);
  const dim3 grid((unsigned)((int64_t)tiles * p.heads)), threads(64 * H::NW);
  if (p.table)
    hipLaunchKernelGGL((tile_kernel<TI, D, true, SPLIT>), grid, threads, 0, s, p, tiles);
  else
    hipLaunchKernelGGL((tile_kernel<TI, D, false, SPLIT>), grid, threads, 0, s, p, tiles);
  return hipGetLastError();
}

template <typename TI, int D>
hipError_t launch_tiles(const AttnParams& p, hipStream_t s) {
  // Few workgroups: keys shared out shorten the chain of tiles.  Measured,
  // split and not, d = 64, 8 heads: 256 tokens 9 and 18 us, 1024 26 and 57, 2048
  // (256 workgroups) 78 and 109, 4096 273 and 260; 16 heads, 1024 49 and 58, 2048
  // 155 and 134.  d = 128, 8 heads: 256 13 and 28, 1024 43 and 97, 2048 142 and 187,
  // 4096 522 and 462; 16 heads, 2048 282 and 235.  d = 256, two waves, one head:
  // 1000 tokens 125 and 169, 3000 362 and 487, 8192 (128 workgroups) 1042 and 1311,
  // two heads of that 2024 and 1318.  With a window of 256, 8 heads, 2048 40 and 23
  // (d = 128 56 and 36), but 512 11.5 and 22 (16 and 35): the rule goes by the window's
  // being there, not by the chains it leaves.
  if (p.window <= 0 && tiles_of(p, 64) * p.heads <= (D == 256 ? 128 : 256)) return launch_tiles<TI, D, true>(p, s);
  return launch_tiles<TI, D, false>(p, s);
}

}  // namespace

int attn_tile_rows(bool bf16_in, int) { return bf16_in ? kPromptRows : 64; }
hipError_t launch_attn_prefill(bool bf16_in, int d, const AttnParams& p, hipStream_t s) {
  if (d == 64) return bf16_in ? launch_prompt<64>(p, s) : launch_tiles<float, 64>(p, s);
  if (d == 128) return bf16_in ? launch_prompt<128>(p, s) : launch_tiles<float, 128>(p, s);
  return bf16_in ? launch_prompt<256>(p, s) : launch_tiles<float, 256>(p, s);
}

// One workgroup on each of 256 compute units.
int attn_decode_waves(bool, int d) { return 256 * (d == 64 ? 8 : d == 128 ? 4 : 2); }
hipError_t launch_attn_decode(bool bf16_in, int d, const AttnParams& p, hipStream_t s) {
  if (d == 64) return bf16_in ? launch_step<bf16, 64>(p, s) : launch_step<float, 64>(p, s);
  if (d == 128) return bf16_in ? launch_step<bf16, 128>(p, s) : launch_step<float, 128>(p, s);
  return bf16_in ? launch_step<bf16, 256>(p, s) : launch_step<float, 256>(p, s);
}

}  // namespace gdn
