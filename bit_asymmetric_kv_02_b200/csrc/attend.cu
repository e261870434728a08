// Attention of one query token per sequence over quantized blocks of R tokens and fp16 residual rows,
// in pages or contiguous, with a sliding window and sinks.
#include <cstdint>

#include "common.cuh"
#include "paged.h"

namespace kivi {
namespace {

// What a sequence of T tokens shows its newest token: t < sink_end or start <= t < T; tokens
// [0, quant) are codes, [quant, T) residual rows.
struct Span {
  int len, quant, start, sink_end;
};
// A length the block table cannot hold counts as 0 (and *bad is set).
__device__ __forceinline__ Span span_of(const AttendArgs& a, int b, bool* bad) {
  Span s;
  *bad = false;
  if (a.lens != nullptr) {
    s.len = __ldg(a.lens + b);
    if (s.len < 0 || (s.len > 0 && ((s.len - 1) >> a.lg_r) > a.max_blocks)) {
      *bad = true;
      s.len = 0;
    }
    s.quant = s.len > 0 ? ((s.len - 1) >> a.lg_r) << a.lg_r : 0;
  } else {
    s.len = a.len;
    s.quant = a.quant;
  }
  s.start = max(0, s.len - a.window);
  s.sink_end = min(a.sinks, s.start);
  return s;
}

constexpr int kThreads = 128;

// grid: x = rows, y = query heads.  A warp's lane holds 4 channels; warps take every fourth token.
template <int BITS>
__global__ void __launch_bounds__(kThreads) attend_simple_kernel(AttendArgs a) {
  constexpr int P = 32 / BITS;
  constexpr uint32_t L = (1u << BITS) - 1;
  __shared__ float sm_m[4], sm_l[4], sm_o[4][kHeadDim];
  const int b = blockIdx.x, hq = blockIdx.y, h = hq / a.gqa, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = 1 << a.lg_r;
  int row = b;
  if (a.cu_tokens != nullptr) {
    if (a.cu_tokens[b + 1] == a.cu_tokens[b]) return;
    row = a.cu_tokens[b + 1] - 1;
  }
  if (row < 0 || row >= a.q_rows) {
    report_status(a.status, KIVI_ERR_INTERNAL);
    return;
  }
  const size_t qoff = (static_cast<size_t>(row) * a.heads * a.gqa + hq) * kHeadDim + 4 * lane;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int i = 0; i < 4; ++i) q[i] = h2f(a.q[qoff + i]);
  bool bad;
  const Span s = span_of(a, b, &bad);
  const int T = s.len;
  if (bad) report_status(a.status, KIVI_ERR_INTERNAL);
  for (int t = warp; t < T; t += 4) {
    if (t >= s.sink_end && t < s.start) continue;
    float k[4], v[4];
    if (t < s.quant) {
      size_t blk;
      if (a.block_table != nullptr) {
        const int j = t >> a.lg_r;
        const int page = j < a.max_blocks ? a.block_table[static_cast<size_t>(b) * a.max_blocks + j] : -1;
        if (page < 0 || page >= a.num_pages) {
          report_status(a.status, KIVI_ERR_INTERNAL);
          continue;
        }
        blk = static_cast<size_t>(page) * a.heads + h;
      } else {
        blk = (static_cast<size_t>(b) * a.heads + h) * a.blocks_per_head + (t >> a.lg_r);
      }
      const int tr = t & (R - 1);
      const uint32_t* kc = a.k_codes + (blk * R + tr) * (kHeadDim / P);
      const uint32_t* vc = a.v_codes + (blk * (R / P) + tr / P) * kHeadDim;
      const float vs = h2f(a.v_scale[blk * (R >> a.lg_gv) + (tr >> a.lg_gv)]);
      const float vz = h2f(a.v_zero[blk * (R >> a.lg_gv) + (tr >> a.lg_gv)]);
      for (int i = 0; i < 4; ++i) {
        const int c = 4 * lane + i;
        const float ks = h2f(a.k_scale[blk * (kHeadDim >> a.lg_gk) + (c >> a.lg_gk)]);
        const float kz = h2f(a.k_zero[blk * (kHeadDim >> a.lg_gk) + (c >> a.lg_gk)]);
        k[i] = static_cast<float>((kc[c / P] >> (BITS * (c % P))) & L) * ks + kz;
        v[i] = static_cast<float>((vc[c] >> (BITS * (tr % P))) & L) * vs + vz;
      }
    } else {
      const size_t off = ((static_cast<size_t>(b) * a.heads + h) * R + (t - s.quant)) * kHeadDim + 4 * lane;
      for (int i = 0; i < 4; ++i) {
        k[i] = h2f(a.k_res[off + i]);
        v[i] = h2f(a.v_res[off + i]);
      }
    }
    float x = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= a.qscale;
    const float mn = fmaxf(m, x), al = exp2f(m - mn), p = exp2f(x - mn);
    l = l * al + p;
    for (int i = 0; i < 4; ++i) o[i] = o[i] * al + p * v[i];
    m = mn;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
  for (int i = 0; i < 4; ++i) sm_o[warp][4 * lane + i] = o[i];
  __syncthreads();
  const int c = threadIdx.x;
  float mm = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3])), num = 0.f, den = 0.f;
  for (int w = 0; w < 4; ++w) {
    if (sm_l[w] == 0.f) continue;
    const float e = exp2f(sm_m[w] - mm);
    num += e * sm_o[w][c];
    den += e * sm_l[w];
  }
  a.out[(static_cast<size_t>(row) * a.heads * a.gqa + hq) * kHeadDim + c] =
      __half_as_ushort(__float2half_rn(den > 0.f ? num / den : (den == 0.f ? 0.f : num)));
}

}  // namespace

size_t attend_workspace_bytes(long long rows, int heads, int gqa) {
  (void)rows, (void)heads, (void)gqa;
  return 256;
}

cudaError_t launch_attend(const AttendArgs& a, int bits, void* workspace, cudaStream_t stream) {
  (void)workspace;
  if (a.rows == 0) return cudaSuccess;
  const dim3 grid(a.rows, a.heads * a.gqa);
  if (bits == 2)
    attend_simple_kernel<2><<<grid, kThreads, 0, stream>>>(a);
  else
    attend_simple_kernel<4><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kivi
