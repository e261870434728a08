// The paged cache's write side: a step's new tokens along the runs that the tables kernel built.
//
// One CTA per (run, KV head, K or V), 2R threads, each holding an 8-token x 8-channel tile of the
// block in registers (quant_tiles.cuh): a block that the step completes is read once - its first rows
// from the residual, where earlier steps left them, the others from the new tokens - and its codes and
// (s, z) come from the same registers.  One pass over the new tokens bounds it.
// A sequence's residual holds its newest block, so the run that completes the block the residual still
// holds part of must read those rows before the sequence's last run overwrites them: the two are
// chained, done by one CTA in that order.
#include <cstdint>

#include "common.cuh"
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
  const int4 a = __ldg(p), b = __ldg(p + 1);
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
}

// grid: x = runs (at most) x KV heads, heads fastest (neighbours in the token-major source); y = K, V;
// block = 2R threads
template <int BITS, int NT>
__global__ void __launch_bounds__(NT) paged_append_kernel(PagedAppendArgs a) {
  constexpr int P = 32 / BITS;
  const int num_runs = min(__ldg(a.counts), a.max_runs);
  int r = static_cast<int>(blockIdx.x / a.heads);
  if (r >= num_runs) return;
  Run run = load_run(a.runs, r);
  if (run.flags & 2) return;  // done by the run that chains to it
  const int h = static_cast<int>(blockIdx.x % a.heads), R = a.residual;
  const bool is_v = blockIdx.y != 0;
  const int c = threadIdx.x & 15, row0 = (threadIdx.x >> 4) * kTileTokens;
  const uint16_t* src = is_v ? a.v : a.k;
  for (;;) {
    if (run.seq < 0 || run.seq >= a.num_seqs || run.page >= a.num_pages || run.page < -1 || run.lo < 0 || run.lo >= run.hi ||
        run.hi > R || run.src < 0 || run.src > a.max_tokens - (run.hi - run.lo)) {
      report_status(a.status, KIVI_ERR_INTERNAL);
      return;
    }
    uint4* res = reinterpret_cast<uint4*>((is_v ? a.v_res : a.k_res) +
                                          (static_cast<size_t>(run.seq) * a.heads + h) * R * kHeadDim);
    const bool last = run.flags & 1;
    const bool whole = run.hi == R && run.page >= 0;
    uint4 x[kTileTokens];
#pragma unroll
    for (int k = 0; k < kTileTokens; ++k) {
      const int row = row0 + k;
      x[k] = make_uint4(0, 0, 0, 0);
      if (row >= run.lo && row < run.hi)
        x[k] = __ldg(reinterpret_cast<const uint4*>(src + (run.src + row - run.lo) * a.token_stride + h * a.head_stride) + c);
      else if (whole && row < run.lo)
        x[k] = res[row * kChunks + c];
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

template <int BITS>
cudaError_t launch(const PagedAppendArgs& a, cudaStream_t stream) {
  const int runs = a.max_runs < a.max_tokens ? a.max_runs : a.max_tokens;  // a run holds at least one new token
  const dim3 grid(static_cast<unsigned>(runs) * a.heads, 2);
  if (a.residual == 128)
    paged_append_kernel<BITS, 256><<<grid, 256, 0, stream>>>(a);
  else if (a.residual == 256)
    paged_append_kernel<BITS, 512><<<grid, 512, 0, stream>>>(a);
  else
    paged_append_kernel<BITS, 1024><<<grid, 1024, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, int bits, cudaStream_t stream) {
  return bits == 2 ? launch<2>(a, stream) : launch<4>(a, stream);
}

}  // namespace kivi
