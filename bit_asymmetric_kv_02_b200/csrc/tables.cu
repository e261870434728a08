// Block tables and slot maps of a paged-cache step, built from request lengths.
//
// Everything is a prefix sum over the rows: new tokens (cu_tokens), blocks that fill (pages from the
// queue's head), pages of finished rows (to the queue's tail) and runs (one per touched block).  Every
// CTA of one cluster scans all rows itself - at most 8192, a few KB from L2 - and then writes its
// share of the tokens, runs, table and ring entries, which it finds by bisection in the prefix sums:
// no CTA waits for another's result.  The cluster barrier at the end only orders the last writes
// (lengths and queue) behind every CTA's reads, so that both may be updated in place.
#include <cstdint>

#include <cooperative_groups.h>

#include "common.cuh"
#include "paged.h"

namespace kivi {
namespace {

namespace cg = cooperative_groups;

constexpr int kTablesThreads = 1024;

struct Sum2 {
  long long a, b;
};
__device__ __forceinline__ Sum2 operator+(Sum2 x, Sum2 y) { return {x.a + y.a, x.b + y.b}; }

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
__device__ Sum2 block_scan(Sum2 v, Sum2* total) {
  __shared__ Sum2 warp_sum[kTablesThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sum2 x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sum2 y = {__shfl_up_sync(0xffffffffu, x.a, off), __shfl_up_sync(0xffffffffu, x.b, off)};
    if (lane >= off) x = x + y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  Sum2 s = warp_sum[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sum2 y = {__shfl_up_sync(0xffffffffu, s.a, off), __shfl_up_sync(0xffffffffu, s.b, off)};
    if (lane >= off) s = s + y;
  }
  *total = {__shfl_sync(0xffffffffu, s.a, 31), __shfl_sync(0xffffffffu, s.b, 31)};
  const int before = warp == 0 ? 0 : warp - 1;
  Sum2 base = {__shfl_sync(0xffffffffu, s.a, before), __shfl_sync(0xffffffffu, s.b, before)};
  if (warp == 0) base = {0, 0};
  __syncthreads();  // warp_sum may be used again
  return {base.a + x.a - v.a, base.b + x.b - v.b};
}

// The row that holds element e of a prefix array of n + 1 entries: first[row] <= e < first[row + 1].
__device__ __forceinline__ int row_of(const int32_t* first, int n, int e) {
  int lo = 0, hi = n;  // first[lo] <= e, and e < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= e)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t clamp32(long long x) {
  return static_cast<int32_t>(x > 0x7fffffffll ? 0x7fffffffll : x);
}

__global__ void __launch_bounds__(kTablesThreads) tables_kernel(TablesArgs a) {
  extern __shared__ int32_t sm[];
  const int n = a.num_rows, tid = threadIdx.x;
  int32_t* cu = sm;               // [n + 1] new tokens
  int32_t* takes = cu + n + 1;    // [n + 1] pages taken
  int32_t* gives = takes + n + 1; // [n + 1] pages given back
  int32_t* nruns = gives + n + 1; // [n + 1] runs
  int32_t* len = nruns + n + 1;   // [n] cached tokens; -1: the row cannot be served
  const int R = 1 << a.lg_r;
  const long long head = a.queue[0], tail = a.queue[1];
  long long avail = tail - head;
  avail = avail < 0 || head < 0 ? 0 : (avail > a.num_pages ? a.num_pages : avail);
  const int per = (n + kTablesThreads - 1) / kTablesThreads;
  const int row0 = min(n, tid * per), row1 = min(n, row0 + per);

  // new tokens and pages each row asks for
  Sum2 mine = {0, 0};
  for (int i = row0; i < row1; ++i) {
    const long long L = a.lens[i], add = max(a.new_tokens[i], 0), end = L + add;
    const bool bad = L < 0 || (L >> a.lg_r) > a.max_blocks || (end >> a.lg_r) > a.max_blocks || end > 0x7fffffffll;
    mine.a += add;
    if (!bad) mine.b += (end >> a.lg_r) - (L >> a.lg_r);
  }
  Sum2 total;
  Sum2 at = block_scan(mine, &total);
  const bool fits = total.a <= a.max_tokens;
  const long long tokens = fits ? total.a : 0;
  // runs and pages given back, of the rows that can be served
  Sum2 work = {0, 0};
  {
    long long asked = at.b, tok = at.a;
    for (int i = row0; i < row1; ++i) {
      const int nt = a.new_tokens[i];
      const long long L = a.lens[i], add = max(nt, 0), end = L + add;
      const bool bad = L < 0 || (L >> a.lg_r) > a.max_blocks || (end >> a.lg_r) > a.max_blocks || end > 0x7fffffffll;
      const long long need = bad ? 0 : (end >> a.lg_r) - (L >> a.lg_r);
      cu[i] = fits ? clamp32(tok) : 0;
      takes[i] = clamp32(min(asked, avail));
      asked += need;
      tok += add;
      const bool ok = fits && !bad && (need == 0 || asked <= avail);
      len[i] = ok ? static_cast<int32_t>(L) : -1;
      gives[i] = clamp32(work.b);
      nruns[i] = clamp32(work.a);
      if (ok && nt > 0) work.a += ((end - 1) >> a.lg_r) - (L >> a.lg_r) + 1;
      if (ok && nt < 0) work.b += L >> a.lg_r;
    }
  }
  Sum2 work_total;
  const Sum2 before = block_scan(work, &work_total);
  for (int i = row0; i < row1; ++i) {
    gives[i] = clamp32(gives[i] + before.b);
    nruns[i] = clamp32(nruns[i] + before.a);
  }
  // pages taken: a row that asks past `avail` takes none, and neither does any later one, so the
  // prefix of the rows served is the prefix of what was asked, up to the first row that fails
  if (tid == 0) {
    cu[n] = static_cast<int32_t>(tokens);
    takes[n] = clamp32(min(total.b, avail));
    gives[n] = clamp32(work_total.b);
    nruns[n] = clamp32(work_total.a);
  }
  __syncthreads();

  cg::cluster_group cluster = cg::this_cluster();
  const int gtid = static_cast<int>(cluster.block_rank()) * kTablesThreads + tid;
  const int nthreads = static_cast<int>(cluster.num_blocks()) * kTablesThreads;
  const unsigned np = static_cast<unsigned>(a.num_pages);
  const unsigned head0 = static_cast<unsigned>(head < 0 ? 0 : head % np), tail0 = static_cast<unsigned>(tail < 0 ? 0 : tail % np);
  const bool lead = cluster.block_rank() == 0;

  for (int i = gtid; i <= n; i += nthreads) a.cu_tokens[i] = cu[i];
  // positions, four tokens a thread
  for (long long t64 = gtid * 4ll; t64 < tokens; t64 += nthreads * 4ll) {
    const int t0 = static_cast<int>(t64);
    int row = row_of(cu, n, t0);
    int32_t p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long t = t64 + j;
      while (row < n - 1 && t >= cu[row + 1]) ++row;
      p[j] = len[row] < 0 ? -1 : len[row] + static_cast<int>(t - cu[row]);
    }
    if (t64 + 4 <= tokens) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(p[0], p[1], p[2], p[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t64 + j < tokens) a.positions[t0 + j] = p[j];
    }
  }
  // runs, and with each completed block its table entry
  const int num_runs = min(nruns[n], a.max_runs);
  for (long long r64 = gtid; r64 < num_runs; r64 += nthreads) {
    const int r = static_cast<int>(r64);
    const int i = row_of(nruns, n, r), k = r - nruns[i], touched = nruns[i + 1] - nruns[i];
    const int L = len[i], have = L >> a.lg_r, b = have + k;
    const long long end = static_cast<long long>(L) + (cu[i + 1] - cu[i]), b0 = static_cast<long long>(b) << a.lg_r;
    const int lo = static_cast<int>(max(static_cast<long long>(L), b0) - b0);
    const int hi = static_cast<int>(min(end, b0 + R) - b0);
    const bool last = k == touched - 1, chained = (L & (R - 1)) != 0 && touched > 1;
    int page = -1;
    if (hi == R) {
      page = a.free_pages[(head0 + static_cast<unsigned>(takes[i] + k)) % np];
      a.block_table[static_cast<size_t>(i) * a.max_blocks + b] = page;
    }
    int4* run = reinterpret_cast<int4*>(a.runs + static_cast<size_t>(r) * 8);
    run[0] = make_int4(i, page, cu[i] + static_cast<int>(b0 + lo - L), lo);
    run[1] = make_int4(hi, (last ? 1 : 0) | (last && chained ? 2 : 0), chained && k == 0 ? touched - 1 : 0, 0);
  }
  // pages of finished rows go behind the tail
  const int given = min(gives[n], a.num_pages);
  for (long long e64 = gtid; e64 < given; e64 += nthreads) {
    const int e = static_cast<int>(e64);
    const int i = row_of(gives, n, e);
    a.free_pages[(tail0 + static_cast<unsigned>(e)) % np] =
        a.block_table[static_cast<size_t>(i) * a.max_blocks + (e - gives[i])];
  }
  cluster.sync();  // every CTA has read the lengths and the queue
  if (!lead) return;
  __shared__ int failed, used;
  if (tid == 0) {
    failed = fits ? 0 : 1;
    used = 0;
  }
  __syncthreads();
  for (int i = row0; i < row1; ++i) {
    const int nt = a.new_tokens[i], L = len[i];
    if (L < 0) {
      failed = 1;
      if (a.lens_out != a.lens) a.lens_out[i] = a.lens[i];
      continue;
    }
    const int add = cu[i + 1] - cu[i];
    a.lens_out[i] = nt < 0 ? 0 : L + add;
    const int need = static_cast<int>(((static_cast<long long>(L) + add) >> a.lg_r) - (L >> a.lg_r));
    if (need > 0) atomicMax(&used, takes[i] + need);
  }
  __syncthreads();
  if (tid == 0) {
    a.queue_out[0] = head + used;
    a.queue_out[1] = tail + given;
    a.counts[0] = num_runs;
    a.counts[1] = static_cast<int32_t>(tokens);
    if (failed) report_status(a.status, KIVI_ERR_CAPACITY);
  }
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
  const size_t smem = (5 * static_cast<size_t>(a.num_rows) + 4) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  const int ctas = a.max_tokens > 4 * kTablesThreads || a.num_rows > kTablesThreads ? 8 : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTablesThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tables_kernel, a);
}

}  // namespace kivi
