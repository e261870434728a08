// Launch arguments of the paged-cache, rotary and windowed-attention kernels (host <-> device).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "kivi.h"

namespace kivi {

constexpr int kMaxPagedSeqs = 8192;  // rows whose prefix sums one CTA keeps in shared memory

struct TablesArgs {
  const int32_t* lens;
  const int32_t* new_tokens;
  int32_t* lens_out;
  int32_t* block_table;
  int32_t* free_pages;
  const int64_t* queue;
  int64_t* queue_out;
  int32_t *cu_tokens, *positions, *runs, *counts;
  int32_t* status;
  int num_rows, num_seqs, max_blocks, num_pages;
  int lg_r;  // log2(residual)
  int max_tokens, max_runs;
};
cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream);

struct RotaryHeads {
  const void* x;
  uint16_t* y;
  const void* weight;
  int heads, rotate;
  long long x_batch, x_token, x_head, y_batch, y_token, y_head;
};
struct RotaryArgs {
  RotaryHeads h[3];  // queries, keys, values
  const int32_t* positions;
  int position0;
  int batch, tokens, heads;  // heads: of all three kinds
  int rotary_dim, interleaved;
  float magnitude, eps;
  uint64_t turns[64];
};
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t stream);

struct PagedAppendArgs {
  const int32_t* runs;    // [max_runs][8]
  const int32_t* counts;  // counts[0] runs
  const uint16_t *k, *v;
  long long token_stride, head_stride;
  uint32_t *k_codes, *v_codes;
  uint16_t *k_scale, *k_zero, *v_scale, *v_zero, *k_res, *v_res;
  int32_t* status;
  int heads, num_pages, num_seqs, residual, lg_gk, lg_gv, max_tokens, max_runs;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, int bits, cudaStream_t stream);

// Attention of one query token per sequence over blocks of R tokens.  Block j of sequence b and KV
// head h is block (page * H + h) of the code and scale arrays, page = block_table[b][j]; without a
// table (the contiguous cache) it is block (b * H + h) * blocks_per_head + j.
struct AttendArgs {
  const uint32_t *k_codes, *v_codes;
  const uint16_t *k_scale, *k_zero, *v_scale, *v_zero, *k_res, *v_res;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* block_table;  // nullptr: contiguous
  const int32_t* lens;         // nullptr: every sequence has `len` tokens, `quant` of them codes
  const int32_t* cu_tokens;    // nullptr: sequence i's query is row i
  const int32_t* positions;    // of the step's plan, or nullptr: a negative one is of a sequence that was not served
  float* partials;
  int32_t* tickets;
  int32_t* status;
  int rows, heads, gqa;
  int max_rows;          // rows the workspace is for
  int passes, per_pass;  // query passes per KV head and queries of a pass (set by launch_attend)
  int len, quant;  // without lens: tokens of every sequence, and how many of them are codes
  int q_rows;
  int max_tokens;  // entries of positions
  int num_pages, max_blocks, blocks_per_head;
  int lg_r, lg_gk, lg_gv;
  int lg_upb;  // log2 of the units per block (set by launch_attend)
  int window, sinks;  // window: INT32_MAX when every token is visible
  float qscale;       // softmax scale * log2(e)
};
constexpr int kAttendResTokens = 16;  // tokens of a residual unit
constexpr int attend_unit_tokens(int bits) { return 256 / bits; }
// max_units: units (of codes and of residual rows) a head can have.  0: more units in all than 32 bits count.
size_t attend_workspace_bytes(long long rows, int heads, int gqa, long long max_units);
cudaError_t launch_attend(AttendArgs a, int bits, void* workspace, cudaStream_t stream);

}  // namespace kivi
