// Tiles in LDS as the scan and the attention keep them: rows in swizzled
// 16-byte granules, read by rows or by columns as MFMA operands, and floats
// split into bf16 terms.
#pragma once

#include "gdn_device.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

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

// The LDS transpose read: lane j of a 16-lane group gets element j % 4 of
// the 8 bytes that lane 4 k + j / 4 names, as its element k.
__device__ __forceinline__ bf16x8 ssm_tr(const char* lo, const char* hi) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)hi);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Columns of x (rows in their own order).
template <typename TI, int P>
struct SsmCols {
  static constexpr int RB = P * (int)sizeof(TI), GR = RB / 16;
  uint32_t at[4];  // bf16: [0]; f32: one for each of four rows
  __device__ __forceinline__ SsmCols(int col0, int lane) {
    const int q = lane >> 4, j = lane & 15;
    if constexpr (sizeof(TI) == 2) {
      const int c = col0 + 4 * (j & 3), r = 4 * q + (j >> 2);
      at[0] = r * RB + (((c >> 3) ^ ssm_swz<GR>(r)) * 16) + (c & 4) * 2;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = col0 + j, r = 4 * q + e;
        at[e] = r * RB + (((c >> 2) ^ ssm_swz<GR>(r)) * 16) + (c & 3) * 4;
      }
    }
  }
  // column col0 + 16 ct + l % 16 over the tokens of unit tu (col0 a multiple
  // of the wave's columns, so that a column tile is an exclusive or)
  __device__ __forceinline__ typename Unit<TI>::type column(const char* tile, int ct, int tu) const {
    if constexpr (sizeof(TI) == 2) {
      const char* a = tile + (at[0] ^ (ct * 32)) + tu * 32 * RB;
      return ssm_tr(a, a + 16 * RB);
    } else {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *(const float*)(tile + (at[e] ^ (ct * 64)) + tu * 16 * RB);
      return v;
    }
  }
};

// Two floats as TERMS packed bf16 pairs (the first in the low half), each
// the rounding of what the ones before leave; a term leaves at most 2^-8 of
// what it rounds, exactly representable as a float.
template <int TERMS>
__device__ __forceinline__ void ssm_terms(float a, float b, uint32_t (&t)[TERMS]) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    bf16x2 v;
    v[0] = (bf16)a;
    v[1] = (bf16)b;
    t[i] = __builtin_bit_cast(uint32_t, v);
    if (i + 1 < TERMS) {
      asm("" : "+v"(t[i]));  // unpacked again below, not rounded a second time
      a -= __uint_as_float(t[i] << 16);
      b -= __uint_as_float(t[i] & 0xffff0000u);
    }
  }
}

// Two accumulator tiles' registers as an operand unit in two terms.
template <bool HALF>
__device__ __forceinline__ void ssm_split2(const f32x4& t0, const f32x4& t1, bf16x8& hi, bf16x8& lo) {
  uint32_t p[4][2];
  ssm_terms<2>(t0[0], t0[1], p[0]);
  ssm_terms<2>(t0[2], t0[3], p[1]);
  if constexpr (!HALF) {
    ssm_terms<2>(t1[0], t1[1], p[2]);
    ssm_terms<2>(t1[2], t1[3], p[3]);
  } else {
    p[2][0] = p[2][1] = p[3][0] = p[3][1] = 0u;
  }
  hi = __builtin_bit_cast(bf16x8, make_uint4(p[0][0], p[1][0], p[2][0], p[3][0]));
  lo = __builtin_bit_cast(bf16x8, make_uint4(p[0][1], p[1][1], p[2][1], p[3][1]));
}

// s_waitcnt's immediate for vmcnt <= n alone.
__host__ __device__ constexpr int ssm_vmcnt(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

}  // namespace gdn
