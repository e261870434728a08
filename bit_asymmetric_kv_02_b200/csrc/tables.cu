// Block tables and slot maps of a paged-cache step, built from request lengths.
//
// Everything is a prefix sum over the rows: new tokens (cu_tokens), blocks that fill (pages from the
// queue's head), pages of finished rows (to the queue's tail) and runs (one per touched block).  Every
// CTA of one cluster scans all rows itself - at most 8192, a few KB from L2 - and then writes its
// share of the tokens, runs, table and ring entries, which it finds by searching the prefix sums:
// no CTA waits for another's result.  The cluster barrier at the end only orders the last writes
// (lengths and queue) behind every CTA's reads, so that both may be updated in place.
//
// Latency bounds it: the loads of lengths and pages (0.7 us each) and the barriers of the scans.  One scan
// takes all four sums as if every row could be served; where one cannot, a second one takes those that depend
// on it.  Small steps take one CTA of eight warps, whose barriers are cheaper.  64 rows of one new token in a graph: 4.7 us,
// 6.5 with eight CTAs of 32 warps; 1000 rows of 250 to 500 new tokens: 15 us, half of them the positions (1.5 MB from eight SMs).
#include <cstdint>

#include <cooperative_groups.h>

#include "common.cuh"
#include "overlap.cuh"
#include "paged.h"

namespace kivi {
namespace {

namespace cg = cooperative_groups;

constexpr int kTablesThreads = 1024;
constexpr unsigned kFull = 0xffffffffu;

// New tokens, pages asked for, runs and pages given back; the last two of rows that are served.
struct Sums {
  long long tokens, pages;
  long long runs, back;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.tokens + y.tokens, x.pages + y.pages, x.runs + y.runs, x.back + y.back};
}
__device__ __forceinline__ Sums up(const Sums& x, int off) {
  return {__shfl_up_sync(kFull, x.tokens, off), __shfl_up_sync(kFull, x.pages, off), __shfl_up_sync(kFull, x.runs, off),
          __shfl_up_sync(kFull, x.back, off)};
}
__device__ __forceinline__ Sums from(const Sums& x, int lane) {
  return {__shfl_sync(kFull, x.tokens, lane), __shfl_sync(kFull, x.pages, lane), __shfl_sync(kFull, x.runs, lane),
          __shfl_sync(kFull, x.back, lane)};
}

// Exclusive prefix of v over the CTA's threads; *total gets the sum.
__device__ Sums block_scan(const Sums& v, Sums* total) {
  __shared__ Sums warp_sum[kTablesThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
  Sums x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sums y = up(x, off);
    if (lane >= off) x = x + y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  Sums s = {0, 0, 0, 0};
  if (lane < nwarps) s = warp_sum[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sums y = up(s, off);
    if (lane >= off) s = s + y;
  }
  *total = from(s, nwarps - 1);
  Sums base = from(s, warp == 0 ? 0 : warp - 1);
  if (warp == 0) base = {0, 0, 0, 0};
  __syncthreads();  // warp_sum may be used again
  return {base.tokens + x.tokens - v.tokens, base.pages + x.pages - v.pages, base.runs + x.runs - v.runs, base.back + x.back - v.back};
}

// The row that holds element e of a prefix array: first[row] <= e < first[row + 1], given first[lo] <= e < first[hi].
__device__ __forceinline__ int row_of(const int32_t* first, int lo, int hi, int e) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= e)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// The same by a whole warp, 32 places at a time.
__device__ __forceinline__ int row_of_warp(const int32_t* first, int n, int e) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const int below = __popc(__ballot_sync(kFull, at < hi && first[at] <= e));  // the places at or before e come first
    lo += below * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Index x of the ring: x mod np, without a 64-bit division for as long as the counters are below 2^32.
__device__ __forceinline__ unsigned ring_place(long long x, unsigned np) {
  if (x < 0) return 0;
  return (x >> 32) == 0 ? static_cast<unsigned>(x) % np : static_cast<unsigned>(x % np);
}

__device__ __forceinline__ int32_t clamp32(long long x) {
  return static_cast<int32_t>(x > 0x7fffffffll ? 0x7fffffffll : x);
}

// A row's share; ok: it can be served as far as its own length goes.
struct RowNeeds {
  long long L, add, pages;
  bool ok;
};
__device__ __forceinline__ RowNeeds needs_of(const TablesArgs& a, int len, int news) {
  RowNeeds r;
  r.L = len;
  r.add = max(news, 0);
  const long long end = r.L + r.add;
  r.ok = len >= 0 && (r.L >> a.lg_r) <= a.max_blocks && (end >> a.lg_r) <= a.max_blocks && end <= 0x7fffffffll;
  r.pages = r.ok ? (end >> a.lg_r) - (r.L >> a.lg_r) : 0;
  return r;
}
__device__ __forceinline__ long long runs_of(const TablesArgs& a, const RowNeeds& r, int news) {
  return news > 0 ? ((r.L + r.add - 1) >> a.lg_r) - (r.L >> a.lg_r) + 1 : 0;
}

__global__ void __launch_bounds__(kTablesThreads) tables_kernel(const __grid_constant__ TablesArgs a) {
  after_previous_kernel();
  extern __shared__ int32_t sm[];
  const int n = a.num_rows, tid = threadIdx.x;
  int32_t* cu = sm;               // [n + 1] new tokens
  int32_t* takes = cu + n + 1;    // [n + 1] pages taken
  int32_t* gives = takes + n + 1; // [n + 1] pages given back
  int32_t* nruns = gives + n + 1; // [n + 1] runs
  int32_t* len = nruns + n + 1;   // [n] cached tokens; -1: the row cannot be served
  int32_t* news = len + n;        // [n] new tokens asked for
  const int R = 1 << a.lg_r;
  const long long head = a.queue[0], tail = a.queue[1];
  const int per = (n + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
  const int row0 = min(n, tid * per), row1 = min(n, row0 + per);

  Sums mine = {0, 0, 0, 0};
  bool bad = false;
  for (int i = row0; i < row1; ++i) {
    const int L = a.lens[i], nt = a.new_tokens[i];
    len[i] = L;
    news[i] = nt;
    const RowNeeds r = needs_of(a, L, nt);
    bad = bad || !r.ok;
    mine.tokens += r.add;
    mine.pages += r.pages;
    mine.runs += r.ok ? runs_of(a, r, nt) : 0;
    mine.back += r.ok && nt < 0 ? r.L >> a.lg_r : 0;
  }
  Sums total;
  Sums at = block_scan(mine, &total);
  long long avail = tail - head;
  avail = avail < 0 || head < 0 ? 0 : (avail > a.num_pages ? a.num_pages : avail);
  const bool fits = total.tokens <= a.max_tokens;
  const long long tokens = fits ? total.tokens : 0;
  const bool all_served = !__syncthreads_or(bad || !fits || total.pages > avail);
  if (!all_served) {  // pages taken: a row that asks past `avail` takes none, and neither does any later one, so the prefix of
                      // the rows served is the prefix of what was asked, up to the first row that fails
    Sums work = {0, 0, 0, 0};
    long long asked = at.pages;
    for (int i = row0; i < row1; ++i) {
      const RowNeeds r = needs_of(a, len[i], news[i]);
      asked += r.pages;
      const bool ok = fits && r.ok && (r.pages == 0 || asked <= avail);
      work.runs += ok ? runs_of(a, r, news[i]) : 0;
      work.back += ok && news[i] < 0 ? r.L >> a.lg_r : 0;
    }
    Sums served;
    const Sums before = block_scan(work, &served);
    at.runs = before.runs;
    at.back = before.back;
    total.runs = served.runs;
    total.back = served.back;
  }
  for (int i = row0; i < row1; ++i) {
    const RowNeeds r = needs_of(a, len[i], news[i]);
    cu[i] = fits ? clamp32(at.tokens) : 0;
    takes[i] = clamp32(min(at.pages, avail));
    nruns[i] = clamp32(at.runs);
    gives[i] = clamp32(at.back);
    at.tokens += r.add;
    at.pages += r.pages;
    const bool ok = all_served || (fits && r.ok && (r.pages == 0 || at.pages <= avail));
    at.runs += ok ? runs_of(a, r, news[i]) : 0;
    at.back += ok && news[i] < 0 ? r.L >> a.lg_r : 0;
    if (!ok) len[i] = -1;
  }
  if (tid == 0) {
    cu[n] = static_cast<int32_t>(tokens);
    takes[n] = clamp32(min(total.pages, avail));
    gives[n] = clamp32(total.back);
    nruns[n] = clamp32(total.runs);
  }
  __syncthreads();

  cg::cluster_group cluster = cg::this_cluster();
  const int gtid = static_cast<int>(cluster.block_rank() * blockDim.x) + tid;
  const int nthreads = static_cast<int>(cluster.num_blocks() * blockDim.x);
  const unsigned np = static_cast<unsigned>(a.num_pages);
  const unsigned head0 = ring_place(head, np), tail0 = ring_place(tail, np);
  const bool lead = cluster.block_rank() == 0;

  for (int i = gtid; i <= n; i += nthreads) a.cu_tokens[i] = cu[i];
  // positions: a warp takes 512 tokens and finds their first and last row together, then four tokens a lane at a time (the
  // search of every lane for itself took 14 us of 1000 prompts of 250 to 500 tokens, bound by instructions)
  for (long long w64 = (gtid >> 5) * 512ll; w64 < tokens; w64 += nthreads * 16ll) {
    const int first = row_of_warp(cu, n, static_cast<int>(w64));
    const int end = static_cast<int>(min(w64 + 512, tokens)), last = row_of_warp(cu, n, end - 1);
    int row = first;
    for (long long t64 = w64 + 4 * (tid & 31); t64 < end; t64 += 128) {
      const int t = static_cast<int>(t64);
      if (row < last && t >= cu[row + 1]) row = row_of(cu, row, last + 1, t);
      const int left = cu[row + 1] - t, at = t - cu[row], L = len[row];
      int4 p = L < 0 ? make_int4(-1, -1, -1, -1) : make_int4(L + at, L + at + 1, L + at + 2, L + at + 3);
      if (left >= 4) {
        *reinterpret_cast<int4*>(a.positions + t) = p;
        continue;
      }
      int32_t q[4] = {p.x, p.y, p.z, p.w};
      int r = row;
#pragma unroll
      for (int j = 1; j < 4; ++j) {  // the row ends within these four
        while (r < last && t + j >= cu[r + 1]) ++r;
        if (r != row) q[j] = len[r] < 0 ? -1 : len[r] + (t + j - cu[r]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t + j < end) a.positions[t + j] = q[j];
    }
  }
  // runs, and with each completed block its table entry
  const int num_runs = min(nruns[n], a.max_runs);
  for (long long r64 = gtid; r64 < num_runs; r64 += nthreads) {
    const int r = static_cast<int>(r64);
    const int i = row_of(nruns, 0, n, r), k = r - nruns[i], touched = nruns[i + 1] - nruns[i];
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
    const int i = row_of(gives, 0, n, e);
    a.free_pages[(tail0 + static_cast<unsigned>(e)) % np] =
        a.block_table[static_cast<size_t>(i) * a.max_blocks + (e - gives[i])];
  }
  cluster.sync();  // every CTA has read the lengths and the queue
  if (!lead) return;
  for (int i = row0; i < row1; ++i) {
    const int nt = news[i], L = len[i];
    if (L >= 0)
      a.lens_out[i] = nt < 0 ? 0 : L + max(nt, 0);
    else if (a.lens_out != a.lens)
      a.lens_out[i] = a.lens[i];
  }
  __shared__ int used;
  if (!all_served) {  // up to the last row that took any
    if (tid == 0) used = 0;
    __syncthreads();
    for (int i = row0; i < row1; ++i) {
      const int pages = len[i] < 0 ? 0 : static_cast<int>(needs_of(a, len[i], news[i]).pages);
      if (pages > 0) atomicMax(&used, takes[i] + pages);
    }
    __syncthreads();
  }
  if (tid == 0) {
    a.queue_out[0] = head + (all_served ? total.pages : used);
    a.queue_out[1] = tail + given;
    a.counts[0] = num_runs;
    a.counts[1] = static_cast<int32_t>(tokens);
    if (!all_served) report_status(a.status, KIVI_ERR_CAPACITY);
  }
}

constexpr size_t tables_smem(int rows) { return (6 * static_cast<size_t>(rows) + 4) * sizeof(int32_t); }
static_assert(tables_smem(kMaxPagedSeqs) + 2 * 1024 <= 232448 - 1024, "a CTA holds 227 KB of shared memory");

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
  const size_t smem = tables_smem(a.num_rows);
  if (smem > 48 * 1024) {  // always to the same limit: it is the function's, and another thread's call may be under way
    const cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(tables_smem(kMaxPagedSeqs)));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  const bool small = a.num_rows <= 256 && a.max_tokens <= 4096;
  const int ctas = small ? 1 : 8;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(small ? 256 : kTablesThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // overlap.cuh
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tables_kernel, a);
}

}  // namespace kivi
