// Parameter blocks and host-side launchers of the operators around a
// recurrent layer's projections: the short convolution, the selective state
// space scan and step, and the residual norm (kernels in gdn_layer.hip and
// gdn_ssm.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace gdn {

// A launch has fewer than 2^32 threads.
constexpr int64_t kLaunchThreads = ((int64_t)1 << 32) - 1;

// gdn_short_conv.
struct ShortConvParams {
  const void* x;         // [T, D], token stride x_st, unit channel stride
  void* out;             // token stride o_st
  const float* w;        // [D][width]
  const float* bias;     // [D] or null
  const void* state_in;  // [n_seq][width - 1][D] or null (zeros)
  void* state_out;       // the same layout or null; may be state_in
  const void* cu;        // packed: [n_seq + 1] int32 or int64 (cu_i64), else null
  int64_t x_st, o_st;
  int32_t cu_i64;
  int32_t n_seq, seq_len;  // uniform: n_seq sequences of seq_len tokens
  int32_t t_total, d, width, silu;
  int64_t first_item, end_item;  // a launch's work items (set by the launcher)
};

// The scan's problem sizes, and the rule that cuts sequences into segments.
struct SsmParams {
  const void* x;      // [T, H, P] strides x_st, x_sh
  const float* dt;    // [T, H] strides dt_st, dt_sh
  const void* b;      // [T, G, N]
  const void* c;
  void* out;          // [T, H, P]
  const float* init;  // [n_seq, H, N, P] or null
  float* final_state; // the same or null
  const float* a_log; // [H] or null (zeros)
  const float* dt_bias;
  const float* d_skip;
  int64_t x_st, x_sh, dt_st, dt_sh, b_st, b_sh, c_st, c_sh, o_st, o_sh;
  int32_t heads, group;  // heads, heads per group
  int32_t unit;          // heads per XCD unit (set by the launcher)
  int32_t softplus;
  // segments: n_seq sequences; uniform ones have seq_len tokens and
  // segs_per_seq segments of seg_len tokens (the last may be shorter), packed
  // ones are read from the table (sequence, first token, length, -1 or 4 times
  // the slot plus 1 for a first segment, 2 for a last one) with
  // seg_off[n_seq + 1] giving each sequence's first segment
  int32_t packed, n_seq, seq_len, seg_len, segs_per_seq, max_segs;
  const int32_t* table;
  const int32_t* seg_off;
  // Where sequences are cut (else null).  A sequence of two or more segments
  // has a slot for each and one more: per slot and head the state before the
  // segment (fragment order, see gdn_ssm.hip), in the last one the last
  // segment's end state, and per slot and head the segment's whole decay.
  // Uniform sequences have segs_per_seq + 1 slots each; of packed ones, cuts
  // is (cut sequences, their segments, 0, 0) and then, for each, (sequence,
  // first slot, segments, 0), and cut_table their segments' rows.
  float* slots;
  float* seg_decay;
  const int32_t* cuts;
  const int32_t* cut_table;
  int32_t max_cuts, max_cut_segs;
};

// The segment table of a packed batch (see SsmParams).
struct SsmTable {
  const void* cu;   // [n_seq + 1] int32 or int64 (cu_i64)
  int32_t* seg_off;
  int32_t* table;
  int32_t* cuts;  // this and the next: null when no sequence is cut
  int32_t* cut_table;
  int32_t cu_i64, n_seq, t_total, seg_len, max_segs, max_cuts, max_cut_segs;
  int32_t round;  // segments whose workgroups take a place in every compute unit
};

// gdn_ssm_decode.
struct SsmStepParams {
  const void* x;
  const float* dt;
  const void* b;
  const void* c;
  float* state;  // [n, H, N, P]
  void* out;
  const float* a_log;
  const float* dt_bias;
  const float* d_skip;
  int64_t x_st, x_sh, dt_st, dt_sh, b_st, b_sh, c_st, c_sh, o_st, o_sh;
  int32_t n, heads, group, softplus;
};

// gdn_add_rms_norm.
struct NormParams {
  const void* x;
  const void* res;   // or null
  const float* w;    // [D] or null
  void* res_out;     // or null
  void* out;         // or null
  uint8_t* out_q;    // e4m3, or null
  float* scales;     // [rows] or [rows][groups]
  int64_t rows, x_st, r_st, ro_st, o_st, q_st;
  int32_t d;
  int32_t groups;    // 0: a scale per row; else ceil(d / 128)
  float eps;
};

hipError_t launch_short_conv(bool bf16, bool vec, const ShortConvParams& p, hipStream_t s);
hipError_t launch_add_rms_norm(bool bf16, bool vec, const NormParams& p, hipStream_t s);

// Segments are multiples of this many tokens (two of the scan's blocks).
constexpr int kSsmBlock = 64;
// Workgroups the scan of a large problem is spread over, and the heads that
// one of them takes.
int ssm_target_groups();
int ssm_group_heads(bool bf16, int p, int group);
hipError_t launch_ssm_table(const SsmTable& p, hipStream_t s);
// The segments' end states and their joining (only when sequences are cut),
// then the scan.
hipError_t launch_ssm_states(bool bf16, int n, int p, const SsmParams& sp, hipStream_t s);
hipError_t launch_ssm_scan(bool bf16, int n, int p, const SsmParams& sp, hipStream_t s);
hipError_t launch_ssm_step(bool bf16, int n, int p, const SsmStepParams& sp, hipStream_t s);

}  // namespace gdn
