// Parameter blocks and host-side launchers of the attention over a paged
// key-value cache: its block tables and slot maps, the store of new rows
// (kernels in gdn_cache.hip), and the attention of prompts and of single
// tokens (gdn_attn.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gdn {

// n / d for 0 <= n < 2^31 and d >= 1 by a multiplication: with s the bits of
// d - 1 and m = floor(2^32 (2^s - d) / d) + 1, n / d = (hi(m n) + n) >> s
// (the sum stays below 2^32).
struct Divide {
  uint32_t d, mul, shift;
};
inline Divide divide_by(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
}

// gdn_cache_plan.
struct PlanParams {
  const int32_t* ctx;    // [n]
  const void* cu;        // [n + 1] int32 or int64 (cu_i64), or null: a token each
  int32_t* table;        // [n][width], row stride table_st
  const int32_t* free;   // [n_free_max]
  const int32_t* n_free; // one value
  int32_t* lens;         // [n], may be ctx
  int64_t* slots;        // [t]
  int32_t* n_free_out;   // one value, may be n_free
  int64_t table_st;
  int32_t cu_i64, n, t, width, free_max;
  Divide page;
};

// gdn_cache_release.
struct ReleaseParams {
  const int32_t* done;  // [n]
  int32_t* lens;        // [n]
  int32_t* table;       // [n][width], row stride table_st
  int32_t* free;        // [free_max]
  int32_t* n_free;
  int64_t table_st;
  int32_t n, width, free_max;
  Divide page;
};

// gdn_cache_store.
struct StoreParams {
  const void* k;  // [t, kv, d], strides in bytes
  const void* v;
  void* k_cache;  // [pages, page, kv, d], strides in bytes
  void* v_cache;
  const int64_t* slots;  // [t]
  int64_t k_st, k_sh, v_st, v_sh;
  int64_t kc_sp, kc_st, kc_sh, vc_sp, vc_st, vc_sh;
  int64_t n_slots;  // pages * page
  int32_t t, kv, row_shift;  // log2 of a row's 16-byte granules
  Divide page;
};

// Attention.  Byte strides throughout.
struct AttnParams {
  const void* q;  // [t, heads, d]
  const void* k;  // table: [pages, page, kv, d]; else [t, kv, d]
  const void* v;
  void* out;      // [t, heads, d]
  int64_t q_st, q_sh, o_st, o_sh;
  int64_t k_sp, k_st, k_sh, v_sp, v_st, v_sh;  // (page,) token, head
  const int32_t* table;  // [n_seq][width], row stride table_st; or null
  const int32_t* lens;   // [n_seq] with a table
  const void* cu;        // packed prompts: [n_seq + 1], else null
  int64_t table_st;
  int32_t cu_i64, n_seq, seq_len, t_total;  // uniform: seq_len tokens each
  int32_t heads, kv, group;                 // group = heads / kv
  int32_t width, pages, max_len;            // max_len = width * page.d
  int32_t window, sinks;                    // window 0: none
  float scale;                              // times log2(e)
  Divide page;
  // gdn_attn_decode: what its parts leave for the join
  float* parts;
  int32_t* chains;
  int32_t waves, waves_log2;  // that share the work, a power of two
  int32_t by_pair;            // chains lie by their pair, else by their first wave
};

hipError_t launch_cache_plan(const PlanParams& p, hipStream_t s);
hipError_t launch_cache_release(const ReleaseParams& p, hipStream_t s);
hipError_t launch_cache_store(const StoreParams& p, hipStream_t s);

// Query rows of one workgroup's tile in the prefill: with them, the tiles of
// the packed batch are at most t_total / rows + n_seq a head.
int attn_tile_rows(bool bf16, int d);
hipError_t launch_attn_prefill(bool bf16, int d, const AttnParams& p, hipStream_t s);

// Waves that gdn_attn_decode spreads its work over, query heads of a key head
// that a wave takes at once, and the floats of one part.
int attn_decode_waves(bool bf16, int d);
constexpr int kDecodeHeads = 16;
constexpr int attn_part_floats(int d) { return kDecodeHeads * (d + 2); }
hipError_t launch_attn_decode(bool bf16, int d, const AttnParams& p, hipStream_t s);

}  // namespace gdn
