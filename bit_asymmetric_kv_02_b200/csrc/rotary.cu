// Norms of queries and keys per head with the position rotation, in one pass, rounded once to the
// fp16 the cache holds.
//
// One memory pass (2 bytes read and written per element) bounds it.  A CTA takes a few tokens: its
// threads first work out the tokens' cosines and sines, one per (token, pair), into shared memory;
// then 8 lanes hold one head row (two 16-byte chunks each, chosen so that a pair's two channels are in
// the same lane for every layout) and a warp passes over 4 head rows at a time.
//
// The angle is exact: turns[i] is a pair's frequency in turns per position as a 64-bit fraction, so
// position * turns[i] modulo 2^64 is the fraction of a turn without any rounding (a float32 product
// would be off by 0.06 rad at position 10^6); its top 32 bits, as a signed number of half turns, go to
// sincospif in fp32.  Norm and rotation are in fp32.
#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"
#include "paged.h"

namespace kivi {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTokens = 4;  // tokens a CTA holds cosines for: one (token, pair) per thread

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

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// grid: x = groups of `per_cta` tokens, y = shares of the heads
template <bool BF16>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryArgs a, int per_cta) {
  __shared__ __align__(16) float2 cs[kRotaryTokens][kHeadDim / 2];
  const int tid = threadIdx.x;
  const unsigned rows = static_cast<unsigned>(a.batch) * a.tokens;  // below 2^31
  const unsigned t0 = blockIdx.x * per_cta;
  const int nt = min(per_cta, static_cast<int>(rows - t0));
  const int pairs = a.rotary_dim / 2;
  {
    const int t = tid >> 6, i = tid & 63;
    if (t < nt && i < pairs) {
      const unsigned row = t0 + t;
      const int pos = a.positions != nullptr ? a.positions[row] : a.position0 + static_cast<int>(row % static_cast<unsigned>(a.tokens));
      const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(pos)) * a.turns[i];
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
      cs[t][i] = make_float2(a.magnitude * c, a.magnitude * s);
    }
  }
  __syncthreads();
  const int j = tid & 7;         // lane of the head row's 8
  const int slot = tid >> 3;     // head row of the CTA's 32
  const int rot = a.rotary_dim / 16;  // lanes whose chunks rotate
  // chunks of 8 channels: the two halves of 8 pairs (half layout), or 8 pairs side by side
  int ca, cb;
  if (a.interleaved || j >= rot) {
    ca = 2 * j;
    cb = 2 * j + 1;
  } else {
    ca = j;
    cb = j + rot;
  }
  const int items = nt * a.heads;
  const int stride = (kRotaryThreads / 8) * gridDim.y;
  for (int it0 = blockIdx.y * (kRotaryThreads / 8); it0 < items; it0 += stride) {
    const int it = it0 + slot;
    const bool live = it < items;
    const int t = live ? it / a.heads : 0;
    int h = live ? it - t * a.heads : 0;
    int kind = 0;
    if (h >= a.h[0].heads) {
      h -= a.h[0].heads;
      kind = 1;
      if (h >= a.h[1].heads) {
        h -= a.h[1].heads;
        kind = 2;
      }
    }
    const RotaryHeads& k = a.h[kind];
    const unsigned row = t0 + t, bu = a.batch == 1 ? 0u : row / static_cast<unsigned>(a.tokens);
    const long long b = bu, ti = row - bu * static_cast<unsigned>(a.tokens);
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(k.x) + b * k.x_batch + ti * k.x_token +
                                                    h * k.x_head);
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    if (live) {
      va = x[ca];
      vb = x[cb];
    }
    float fa[8], fb[8];
    unpack8<BF16>(va, fa);
    unpack8<BF16>(vb, fb);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += fa[i] * fa[i] + fb[i] * fb[i];
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (!live) continue;
    if (k.weight != nullptr) {
      const float r = rsqrtf(sum * (1.0f / kHeadDim) + a.eps);
      const uint4* w = static_cast<const uint4*>(k.weight);
      float wa[8], wb[8];
      unpack8<BF16>(__ldg(w + ca), wa);
      unpack8<BF16>(__ldg(w + cb), wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        fa[i] *= r * wa[i];
        fb[i] *= r * wb[i];
      }
    }
    if (k.rotate && j < rot) {
      const float4* c4 = reinterpret_cast<const float4*>(&cs[t][8 * j]);
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float4 p = c4[i / 2], q = c4[2 + i / 2];  // (cos, sin) of two pairs each
          const float a0 = fa[2 * i], a1 = fa[2 * i + 2], b0 = fb[2 * i], b1 = fb[2 * i + 2];
          fa[2 * i] = a0 * p.x - fa[2 * i + 1] * p.y;
          fa[2 * i + 1] = a0 * p.y + fa[2 * i + 1] * p.x;
          fa[2 * i + 2] = a1 * p.z - fa[2 * i + 3] * p.w;
          fa[2 * i + 3] = a1 * p.w + fa[2 * i + 3] * p.z;
          fb[2 * i] = b0 * q.x - fb[2 * i + 1] * q.y;
          fb[2 * i + 1] = b0 * q.y + fb[2 * i + 1] * q.x;
          fb[2 * i + 2] = b1 * q.z - fb[2 * i + 3] * q.w;
          fb[2 * i + 3] = b1 * q.w + fb[2 * i + 3] * q.z;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float4 p = c4[i / 2];
          const float a0 = fa[i], a1 = fa[i + 1];
          fa[i] = a0 * p.x - fb[i] * p.y;
          fb[i] = a0 * p.y + fb[i] * p.x;
          fa[i + 1] = a1 * p.z - fb[i + 1] * p.w;
          fb[i + 1] = a1 * p.w + fb[i + 1] * p.z;
        }
      }
    }
    uint4* y = reinterpret_cast<uint4*>(k.y + b * k.y_batch + ti * k.y_token + h * k.y_head);
    y[ca] = pack8(fa);
    y[cb] = pack8(fb);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.batch) * a.tokens;
  if (rows == 0 || a.heads == 0) return cudaSuccess;
  // few tokens: one per CTA and the heads split, so that a decode step's rows are all in flight at once
  const bool few = rows < 4 * 148;
  const int per_cta = few ? 1 : kRotaryTokens;
  dim3 grid(static_cast<unsigned>((rows + per_cta - 1) / per_cta), few ? (a.heads + 31) / 32 : 1);
  if (dtype == KIVI_DTYPE_BF16)
    rotary_kernel<true><<<grid, kRotaryThreads, 0, stream>>>(a, per_cta);
  else
    rotary_kernel<false><<<grid, kRotaryThreads, 0, stream>>>(a, per_cta);
  return cudaGetLastError();
}

}  // namespace kivi
