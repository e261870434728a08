// The paged cache's write side: a step's new tokens along the runs that the tables kernel built.
//
// One CTA per (run, KV head, K or V), 2R threads, each holding an 8-token x 8-channel tile of the
// block in registers (quant_tiles.cuh): a block that the step completes is read once - its first rows
// from the residual, where earlier steps left them, the others from the new tokens - and its codes and
// (s, z) come from the same registers.  One pass over the new tokens bounds it: 4 prompts of up to 32768
// tokens x 32 heads (1.72 GB) take 326 us, 298 on other GPUs: 82% to 89% of the copy bandwidth, at 4 bits 65%: its codes
// take half as many instructions again, and a branch each.  A step of 64 single tokens x 32 heads,
// 16 of which complete a block, takes 12.3 us against 6.5 us for its bytes: the launch, the plan, a search in it and two rounds of
// loads that depend on one another.
// A sequence's residual holds its newest block, so the run that completes the block the residual still
// holds part of must read those rows before the sequence's last run overwrites them: the two are
// chained, done by one CTA in that order.
#include <cstdint>

#include "common.cuh"
#include "overlap.cuh"
#include "paged.h"
#include "quant_rules.cuh"
#include "quant_tiles.cuh"

namespace kivi {
namespace {

struct Run {
  int seq, page, src, lo, hi, flags, chain;
};

__device__ __forceinline__ Run load_run(const int32_t* runs, int r) {
  const int4* p = reinterpret_cast<const int4*>(runs) + 2 * static_cast<size_t>(r);
  const int4 a = p[0], b = p[1];
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
}

// 64 registers a thread, so that four blocks of 128 tokens are on an SM and one's loads cover another's codes: a prompt of 4 x 32768
// tokens x 32 heads takes 300 us, 347 with three and 460 with two on the same GPU; 2 x 16000 at 4 bits 146, 172 and 231.
constexpr int kThreadsPerSm = 1024;

// Inside the cache and the source.
__device__ __forceinline__ bool run_ok(const PagedAppendArgs& a, const Run& r, int R) {
  return r.seq >= 0 && r.seq < a.num_seqs && r.page < a.num_pages && r.page >= -1 && r.lo >= 0 && r.lo < r.hi && r.hi <= R &&
         r.src >= 0 && r.src <= a.max_tokens - (r.hi - r.lo);
}

// A run that completes no block and has few rows takes a CTA for kRowHeads heads, K and V both; a longer one goes the way of the
// blocks, a CTA per head and K or V, which has all its rows on the way at once.  More than 16 rows: 64 sequences of up to 16 new
// tokens x 32 heads 12.3 us, 18.0 with 8 here (R = 256: 9.1 and 33); 4 of up to 300 x 32 heads, R = 256, 7.8, 13.0 with 32 here.  What
// loses is 100 of up to 24 x 8 heads: 8.9, 7.4 with 32 (R = 512: 27 and 7.4).
constexpr int kFewRows = 16;
__device__ __forceinline__ bool few_rows(const Run& r) { return r.page < 0 && r.chain == 0 && r.hi - r.lo <= kFewRows; }

// A run of few rows: one CTA takes its residual rows of kRowHeads heads from h on, K and V both.
template <int NT>
__device__ __forceinline__ void append_rows(const PagedAppendArgs& a, const Run& run, int h) {
  constexpr int R = NT / 2;
  if (!run_ok(a, run, R)) {
    report_status(a.status, KIVI_ERR_INTERNAL);
    return;
  }
  const int c = threadIdx.x & 15, hh = h + (threadIdx.x >> 4);
  if (hh >= a.heads || !(run.flags & 1)) return;
  const long long from = run.src * a.token_stride + hh * a.head_stride;
  const size_t to = ((static_cast<size_t>(run.seq) * a.heads + hh) * R + run.lo) * kChunks + c;
  uint4 *kr = reinterpret_cast<uint4*>(a.k_res) + to, *vr = reinterpret_cast<uint4*>(a.v_res) + to;
  const int rows = run.hi - run.lo;
#pragma unroll 1
  for (int i0 = 0; i0 < rows; i0 += 4) {  // four rows on their way at once
    uint4 k[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= rows) break;
      k[i] = *(reinterpret_cast<const uint4*>(a.k + from + (i0 + i) * a.token_stride) + c);
      v[i] = *(reinterpret_cast<const uint4*>(a.v + from + (i0 + i) * a.token_stride) + c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= rows) break;
      kr[(i0 + i) * kChunks] = k[i];
      vr[(i0 + i) * kChunks] = v[i];
    }
  }
}

// A run that completes a block, or the chain of runs that begins with it: one CTA per head and K or V.  FRESH: blocks of new tokens
// alone, most of a prompt's, take loads without the choice of place, 150 of the 384 logic instructions a thread: 4 prompts of up to
// 32768 tokens x 32 heads 328 -> 298 us on one GPU, 358 -> 321 on another; 4 x 6000 94 -> 84; 4 bits 2 x 16000 156 -> 147.  A step of few
// tokens has next to none and is 0.5 us slower with the second copy of the loads.
template <int BITS, int NT, bool FRESH>
__device__ __forceinline__ void append_block(const PagedAppendArgs& a, Run run, int r, int num_runs, int h, bool is_v) {
  constexpr int P = 32 / BITS, R = NT / 2;
  const int c = threadIdx.x & 15, row0 = (threadIdx.x >> 4) * kTileTokens;
  const uint16_t* src = is_v ? a.v : a.k;
  for (;;) {
    if (!run_ok(a, run, R)) {
      report_status(a.status, KIVI_ERR_INTERNAL);
      return;
    }
    uint4* res = reinterpret_cast<uint4*>((is_v ? a.v_res : a.k_res) +
                                          (static_cast<size_t>(run.seq) * a.heads + h) * R * kHeadDim);
    const bool last = run.flags & 1;
    const bool whole = run.hi == R && run.page >= 0;
    const int skip = whole ? 0 : run.lo;  // rows before it are not looked at
    const char* fresh = reinterpret_cast<const char*>(src + (run.src - run.lo) * a.token_stride + h * a.head_stride) + 16 * c;
    const char* old = reinterpret_cast<const char*>(res) + 16 * c;
    uint4 x[kTileTokens];
    if (FRESH && whole && run.lo == 0) {
#pragma unroll
      for (int k = 0; k < kTileTokens; ++k) x[k] = *reinterpret_cast<const uint4*>(fresh + (row0 + k) * a.token_stride * 2);
    } else {
#pragma unroll
      for (int k = 0; k < kTileTokens; ++k) {  // one load per row, from either place
        const int row = row0 + k;
        const char* at = row >= run.lo ? fresh + row * a.token_stride * 2 : old + row * (kHeadDim * 2);
        x[k] = make_uint4(0, 0, 0, 0);
        if (row >= skip && row < run.hi) x[k] = *reinterpret_cast<const uint4*>(at);
      }
    }
    if (last) {
#pragma unroll
      for (int k = 0; k < kTileTokens; ++k)
        if (row0 + k >= run.lo && row0 + k < run.hi) res[(row0 + k) * kChunks + c] = x[k];
    }
    if (whole) {
      const size_t blk = static_cast<size_t>(run.page) * a.heads + h;
      if (!is_v)
        quantize_k_tiles<BITS>(x, a.lg_gk, a.k_codes + blk * R * (kHeadDim / P), a.k_scale + blk * (kHeadDim >> a.lg_gk),
                               a.k_zero + blk * (kHeadDim >> a.lg_gk), false);
      else
        quantize_v_tiles<BITS>(x, R, a.lg_gv, a.v_codes + blk * (R / P) * kHeadDim, a.v_scale + blk * (R >> a.lg_gv),
                               a.v_zero + blk * (R >> a.lg_gv));
    }
    if (run.chain == 0) return;
    __syncthreads();  // the residual rows have been read, and the tile code's shared memory is free again
    r += run.chain;
    if (run.chain < 0 || r >= num_runs) {
      report_status(a.status, KIVI_ERR_INTERNAL);
      return;
    }
    run = load_run(a.runs, r);
    run.chain = 0;
  }
}

// Runs of the plan that are looked at.
__device__ __forceinline__ int runs_of(const PagedAppendArgs& a, const int2& counts, bool reports) {
  if (reports && (counts.x > a.max_runs || counts.y > a.max_tokens))
    report_status(a.status, KIVI_ERR_INTERNAL);  // a plan of more than the source or its own arrays hold: what fits is done
  return min(counts.x, a.max_runs);
}

// grid: x = runs (at most) x KV heads, heads fastest (neighbours in the token-major source); y = K, V; block = 2R threads.
template <int BITS, int NT>
__global__ void __launch_bounds__(NT, kThreadsPerSm / NT) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  after_previous_kernel();
  constexpr int kRowHeads = NT / 16;
  const int r = static_cast<int>(blockIdx.x / a.heads), h = static_cast<int>(blockIdx.x % a.heads);
  const Run run = load_run(a.runs, r);  // r < max_runs: the plan holds that many, used or not
  const int num_runs = runs_of(a, *reinterpret_cast<const int2*>(a.counts), r == 0);
  if (r >= num_runs || (run.flags & 2)) return;  // flag 2: done by the run that chains to it
  if (!few_rows(run))
    append_block<BITS, NT, true>(a, run, r, num_runs, h, blockIdx.y != 0);
  else if (blockIdx.y == 0 && h % kRowHeads == 0)
    append_rows<NT>(a, run, h);
}

// The same for at most NT runs few of which complete a block: the grid fills the SMs once, and its CTAs go through the work that
// there is, which each counts for itself.
template <int BITS, int NT>
__global__ void __launch_bounds__(NT, kThreadsPerSm / NT) paged_append_few_kernel(const __grid_constant__ PagedAppendArgs a) {
  after_previous_kernel();
  constexpr int kRowHeads = NT / 16;
  __shared__ int warp_sum[NT / 32], found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Run mine{};
  if (tid < a.max_runs) mine = load_run(a.runs, tid);
  const int num_runs = min(NT, runs_of(a, *reinterpret_cast<const int2*>(a.counts), blockIdx.x == 0));
  int work = 0;
  if (tid < num_runs && !(mine.flags & 2)) work = few_rows(mine) ? (a.heads + kRowHeads - 1) / kRowHeads : 2 * a.heads;
  int before = work;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += y;
  }
  if (lane == 31) warp_sum[warp] = before;
  __syncthreads();
  before -= work;
  int total = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    if (i < warp) before += warp_sum[i];
    total += warp_sum[i];
  }
  for (int item = static_cast<int>(blockIdx.x); item < total; item += static_cast<int>(gridDim.x)) {
    if (item >= before && item < before + work) {
      found[0] = tid;
      found[1] = item - before;
    }
    __syncthreads();
    const int r = found[0], i = found[1];
    const Run run = load_run(a.runs, r);
    if (few_rows(run))
      append_rows<NT>(a, run, i * kRowHeads);
    else
      append_block<BITS, NT, false>(a, run, r, num_runs, i >> 1, i & 1);
    __syncthreads();
  }
}

template <int BITS, int NT>
cudaError_t launch_tiles(const PagedAppendArgs& a, cudaStream_t stream) {
  // a run holds at least one new token; without any, one block looks whether the plan says so too
  const int runs = max(1, min(a.max_runs, a.max_tokens));
  const long long ctas = 2ll * runs * a.heads;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // Few of the runs complete a block when there are few tokens to a run: then most of a grid of all runs x heads finds nothing to
  // do, and a grid that fills the SMs once takes over, if that one does not.  32 heads, that grid against this one: 64 single
  // tokens 14.1 -> 12.5 us (R = 256 27.8 -> 24.2, R = 512 60.5 -> 54.3), 16 at R = 512 17.0 -> 13.5, 64 x up to 60 at R = 512 105.7 ->
  // 79.7; but 4 prompts of up to 300 tokens 7.4 -> 9.1 and of up to 6000 84 -> 116, where blocks that start as others end keep the SMs
  // fuller.  The rule gives 64 x up to 16 the wrong one at R = 128 (10.5 -> 12.3) and the right one at R = 256 (18.9 -> 9.1).
  const int slots = sms * (kThreadsPerSm / NT);
  if (runs <= NT && a.max_tokens < runs * (NT / 8) && ctas > slots)
    return launch_overlapped(paged_append_few_kernel<BITS, NT>, dim3(slots), NT, 0, stream, a);
  return launch_overlapped(paged_append_kernel<BITS, NT>, dim3(static_cast<unsigned>(runs) * a.heads, 2), NT, 0, stream, a);
}
template <int BITS>
cudaError_t launch(const PagedAppendArgs& a, cudaStream_t stream) {
  if (a.residual == 128) return launch_tiles<BITS, 256>(a, stream);
  if (a.residual == 256) return launch_tiles<BITS, 512>(a, stream);
  return launch_tiles<BITS, 1024>(a, stream);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int bits, cudaStream_t stream) {
  return bits == 2 ? launch<2>(a, stream) : launch<4>(a, stream);
}

}  // namespace kivi
