// Norms of queries and keys per head with the position rotation, in one pass, rounded once to the
// fp16 the cache holds.
//
// One memory pass (2 bytes read and written per element) bounds it.  A warp takes a token and its heads,
// four head rows at a time: 8 lanes hold one head row (two 16-byte chunks each, chosen so that a pair's two
// channels are in the same lane for every layout).  The token's cosines and sines are formed once, two pairs
// a lane, and stay in registers with the norm's weights multiplied in, four factors a pair.  The rows of the
// next four steps are on their way to shared memory meanwhile: 32768 tokens x 40 heads in bf16 take 120 us,
// 108 on other GPUs, 86% to 96% of the copy bandwidth; with one step ahead in registers (24 KB in flight per SM) 141 us, and with
// blocks of four tokens that read their cosines from shared memory for every head 145 us.
//
// The angle is exact: turns[i] is a pair's frequency in turns per position as a 64-bit fraction, so
// position * turns[i] modulo 2^64 is the fraction of a turn without any rounding (a float32 product
// would be off by 0.06 rad at position 10^6); its top 32 bits, as a signed number of half turns, go to
// sincospif in fp32.  Norm and rotation are in fp32.
#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"
#include "overlap.cuh"
#include "paged.h"

namespace kivi {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryWarps = kRotaryThreads / 32;
constexpr int kRowsAtOnce = 4;  // head rows a warp holds
constexpr int kDepth = 4;       // steps whose rows are on their way

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<BF16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// grid: x = groups of 8 tokens, y = shares of `share` heads of all kinds
template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads, 3) rotary_kernel(const __grid_constant__ RotaryArgs a, int share) {
  __shared__ __align__(16) float2 cs[kRotaryWarps][kHeadDim / 2];
  __shared__ uint4 ring[kRotaryWarps][kDepth][2][32];  // a lane's two chunks of the head rows on their way
  after_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned row = blockIdx.x * kRotaryWarps + warp;
  if (row >= static_cast<unsigned>(a.batch) * a.tokens) return;  // below 2^31
  const unsigned bu = a.batch == 1 ? 0u : row / static_cast<unsigned>(a.tokens);
  const long long b = bu, ti = row - bu * static_cast<unsigned>(a.tokens);
  const int j = lane & 7, slot = lane >> 3;
  const int pairs = a.rotary_dim / 2, rot = a.rotary_dim / 16;  // lanes j < rot hold pairs 8 j .. 8 j + 7
  // chunks of 8 channels: the two halves of 8 pairs (half layout), or 8 pairs side by side
  const bool apart = !INTERLEAVED && j < rot;
  const int ca = apart ? j : 2 * j, cb = apart ? j + rot : 2 * j + 1;
  const int h1 = min(a.heads, static_cast<int>(blockIdx.y + 1) * share);
  int h = static_cast<int>(blockIdx.y) * share + slot;

  auto kind_of = [&](int at) { return at < a.h[0].heads ? 0 : (at < a.h[0].heads + a.h[1].heads ? 1 : 2); };
  auto index_of = [&](int at, int kind) -> long long {
    return at - (kind > 0 ? a.h[0].heads : 0) - (kind > 1 ? a.h[1].heads : 0);
  };
  const uint32_t mine = smem_u32(&ring[warp][0][0][lane]);
  int ahead = h, put = 0;  // the head row that is fetched next, and its place in the ring
  auto fetch = [&]() {
    if (ahead < h1) {
      const int kind = kind_of(ahead);
      const RotaryHeads& k = a.h[kind];
      const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(k.x) + b * k.x_batch + ti * k.x_token +
                                                      index_of(ahead, kind) * k.x_head);
      copy16(mine + put * 1024, x + ca);
      copy16(mine + put * 1024 + 512, x + cb);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += kRowsAtOnce;
    put = put + 1 == kDepth ? 0 : put + 1;
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) fetch();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = 2 * lane + e;
    if (i < pairs) {
      const int pos = a.positions != nullptr ? a.positions[row] : a.position0 + static_cast<int>(ti);
      const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(pos)) * a.turns[i];
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
      // vector (i / 2) % 4 of lane i / 8: lanes read neighbouring vectors
      cs[warp][2 * (8 * ((i >> 1) & 3) + (i >> 3)) + (i & 1)] = make_float2(a.magnitude * c, a.magnitude * s);
    }
  }
  __syncwarp();
  // first element a, second element b of pair p: a' = a fa - b fb, b' = a ga + b gb; no pair: a' = a fa, b' = b gb
  float fa[8], fb[8], ga[8], gb[8];
  int kind = -1;
  const int steps = (h1 - static_cast<int>(blockIdx.y) * share + kRowsAtOnce - 1) / kRowsAtOnce;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const bool live = h < h1;
    const int now = live ? kind_of(h) : kind;
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");  // a lane reads what it has copied itself
    const uint4 va = ring[warp][put][0][lane], vb = ring[warp][put][1][lane];
    fetch();
    if (live && now != kind) {  // another kind of heads: its factors
      kind = now;
      const uint4* w = static_cast<const uint4*>(a.h[kind].weight);
      float wa[8], wb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.f;
      if (w != nullptr) {
        unpack8<BF16>(w[ca], wa);
        unpack8<BF16>(w[cb], wb);
      }
      const float4* c4 = reinterpret_cast<const float4*>(cs[warp]) + j;
#pragma unroll
      for (int p = 0; p < 8; p += 2) {
        float4 u = make_float4(1.f, 0.f, 1.f, 0.f);  // (cos, sin) of two pairs
        if (a.h[kind].rotate && j < rot) u = c4[4 * p];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int q = p + e;
          const float w0 = INTERLEAVED ? (q < 4 ? wa[2 * q] : wb[2 * q - 8]) : wa[q];
          const float w1 = INTERLEAVED ? (q < 4 ? wa[2 * q + 1] : wb[2 * q - 7]) : wb[q];
          const float c = e ? u.z : u.x, s = e ? u.w : u.y;
          fa[q] = w0 * c;
          fb[q] = w1 * s;
          ga[q] = w0 * s;
          gb[q] = w1 * c;
        }
      }
    }
    float xa[8], xb[8];
    unpack8<BF16>(va, xa);
    unpack8<BF16>(vb, xb);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += xa[i] * xa[i] + xb[i] * xb[i];
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (live) {
      if (a.h[kind].weight != nullptr) {
        const float f = rsqrtf(sum * (1.0f / kHeadDim) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xa[i] *= f;
          xb[i] *= f;
        }
      }
      const bool turned = a.h[kind].rotate && j < rot;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float& x0 = INTERLEAVED ? (q < 4 ? xa[2 * q] : xb[2 * q - 8]) : xa[q];
        float& x1 = INTERLEAVED ? (q < 4 ? xa[2 * q + 1] : xb[2 * q - 7]) : xb[q];
        const float y0 = x0 * fa[q], y1 = x1 * gb[q];  // an infinite element without a partner stays by itself
        const float z0 = turned ? fmaf(-x1, fb[q], y0) : y0;
        x1 = turned ? fmaf(x0, ga[q], y1) : y1;
        x0 = z0;
      }
      const RotaryHeads& k = a.h[kind];
      uint4* y = reinterpret_cast<uint4*>(k.y + b * k.y_batch + ti * k.y_token + index_of(h, kind) * k.y_head);
      y[ca] = pack8(xa);
      y[cb] = pack8(xb);
    }
    h += kRowsAtOnce;
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.batch) * a.tokens;
  if (rows == 0 || a.heads == 0) return cudaSuccess;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // a warp takes all heads of a token where that fills the GPU (16 warps an SM); else the heads are shared out, down to four a
  // warp, so that a decode step's rows are all in flight at once
  const long long want = sms * 16ll;
  long long share = (a.heads * rows + want - 1) / want;
  share = (share + kRowsAtOnce - 1) / kRowsAtOnce * kRowsAtOnce;
  if (share > a.heads) share = a.heads;
  const dim3 grid(static_cast<unsigned>((rows + kRotaryWarps - 1) / kRotaryWarps), static_cast<unsigned>((a.heads + share - 1) / share));
  const int n = static_cast<int>(share);
  const bool bf16 = dtype == KIVI_DTYPE_BF16, side = a.interleaved != 0;
  auto* kernel = bf16 ? (side ? rotary_kernel<true, true> : rotary_kernel<true, false>)
                      : (side ? rotary_kernel<false, true> : rotary_kernel<false, false>);
  return launch_overlapped(kernel, grid, kRotaryThreads, 0, stream, a, n);
}

}  // namespace kivi
