// Register-staged blocks (R <= 512): a CTA of 2R threads reads its block from HBM once.  Thread
// (token group tg = tid / 16, chunk c = tid % 16) holds tokens 8 tg .. 8 tg + 7 x channels 8 c .. 8 c + 7 in registers.
// Every K group (g_k >= 32 channels) and every V group (g_v >= 32 tokens) is a union of whole
// thread tiles, so a thread quantizes its 64 values with one (s, z).  Group extremes travel as the
// fp16 pair (min, -max), which one packed minimum reduces.  The caller loads the tiles (x[k]: token 8 tg + k).
//
// Shared by the prefill, flush and paged append kernels; quant_rules.cuh has the code rule.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "common.cuh"
#include "quant_rules.cuh"

namespace kivi {
namespace {

constexpr int kChunks = kHeadDim / 8;  // uint4 chunks per token row
constexpr int kTileTokens = 8;

__device__ __forceinline__ __half2 tile_min_negmax(const uint4 (&x)[kTileTokens]) {
  __half2 lo = *reinterpret_cast<const __half2*>(&x[0].x), hi = lo;
#pragma unroll
  for (int k = 0; k < kTileTokens; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = *reinterpret_cast<const __half2*>(&w[i]);
      lo = __hmin2(lo, v);
      hi = __hmax2(hi, v);
    }
  }
  return __halves2half2(__hmin(__low2half(lo), __high2half(lo)), __hneg(__hmax(__low2half(hi), __high2half(hi))));
}

__device__ __forceinline__ __half2 shfl_xor_h2(__half2 v, int off) {
  const uint32_t u = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&v), off);
  return *reinterpret_cast<const __half2*>(&u);
}

__device__ __forceinline__ GroupParams group_from_pair(__half2 m, int levels) {
  return make_group(__low2float(m), -__high2float(m), levels);
}

template <int BITS>
__device__ __forceinline__ void quantize_k_tiles(const uint4 (&x)[kTileTokens], int lg_gk, uint32_t* __restrict__ codes,
                                                 uint16_t* __restrict__ scale, uint16_t* __restrict__ zero,
                                                 bool given) {
  constexpr int L = (1 << BITS) - 1;
  __shared__ __half2 red[1024 / 32][kHeadDim / 32];
  __shared__ GroupParams grp[kHeadDim / 32];
  __shared__ Thresh2 thr[kHeadDim / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
  const int c = tid & 15, tg = tid >> 4;

  // K group of chunk c: chunks [cpg * g, cpg * (g + 1)), cpg = g_k / 8; the warp's two token
  // groups (lanes < 16 and >= 16) hold the same chunks
  const int lg_cpg = lg_gk - 3, ngk = kHeadDim >> lg_gk;
  if (!given) {
    __half2 m = tile_min_negmax(x);
    for (int off = 1; off < (1 << lg_cpg); off <<= 1) m = __hmin2(m, shfl_xor_h2(m, off));
    m = __hmin2(m, shfl_xor_h2(m, 16));
    if (lane < 16 && (c & ((1 << lg_cpg) - 1)) == 0) red[warp][c >> lg_cpg] = m;
    __syncthreads();
  }
  if (tid < ngk) {
    GroupParams gp;
    if (given) {  // prefix groups: (s, z) already stored for this block
      gp = group_from_stored(scale[tid], zero[tid]);
    } else {
      __half2 t = red[0][tid];
      for (int w = 1; w < nwarps; ++w) t = __hmin2(t, red[w][tid]);
      gp = group_from_pair(t, L);
      scale[tid] = gp.s_bits;
      zero[tid] = gp.z_bits;
    }
    if constexpr (BITS == 2)
      thr[tid] = make_thresh2(gp);
    else
      grp[tid] = gp;
  }
  __syncthreads();
  const int tok0 = tg * kTileTokens;
  if constexpr (BITS == 4) {  // K word c of a token is exactly the tile's 8 channels
    const GroupParams g = grp[c >> lg_cpg];
#pragma unroll
    for (int k = 0; k < kTileTokens; ++k) codes[(tok0 + k) * (kHeadDim / 8) + c] = quantize_row8<4>(x[k], g);
  } else {  // K word c / 2 of a token: chunk 2i in bits 0..15, chunk 2i + 1 in bits 16..31
    const Thresh2 t = thr[c >> lg_cpg];
    uint32_t h[kTileTokens];
#pragma unroll
    for (int k = 0; k < kTileTokens; ++k) h[k] = row_codes2(x[k], t);
    const bool odd = c & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // the even chunk stores tokens 0..3 of the tile, the odd one 4..7
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? h[j] : h[4 + j], 1);
      const int k = odd ? 4 + j : j;
      const uint32_t word = odd ? (other | (h[4 + j] << 16)) : (h[j] | (other << 16));
      codes[(tok0 + k) * (kHeadDim / 16) + (c >> 1)] = word;
    }
  }
}

template <int BITS>
__device__ __forceinline__ void quantize_v_tiles(const uint4 (&x)[kTileTokens], int R, int lg_gv,
                                                 uint32_t* __restrict__ codes, uint16_t* __restrict__ scale,
                                                 uint16_t* __restrict__ zero) {
  constexpr int L = (1 << BITS) - 1;
  __shared__ __half2 red[1024 / 32];
  __shared__ GroupParams grp[512 / 32];
  __shared__ Thresh2 thr[512 / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = tid & 15, tg = tid >> 4;

  // a warp's 16 tokens lie in one V group (g_v >= 32); group j spans warps [j g_v / 16, ...)
  __half2 m = tile_min_negmax(x);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) m = __hmin2(m, shfl_xor_h2(m, off));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  const int ngv = R >> lg_gv, wpg = 1 << (lg_gv - 4);
  if (tid < ngv) {
    __half2 t = red[tid * wpg];
    for (int w = 1; w < wpg; ++w) t = __hmin2(t, red[tid * wpg + w]);
    const GroupParams gp = group_from_pair(t, L);
    if constexpr (BITS == 2)
      thr[tid] = make_thresh2(gp);
    else
      grp[tid] = gp;
    scale[tid] = gp.s_bits;
    zero[tid] = gp.z_bits;
  }
  __syncthreads();
  const int gv = (tg * kTileTokens) >> lg_gv;
  // codes of channel 8 c + e for the tile's 8 tokens, token k at bits BITS * k
  uint32_t col[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if constexpr (BITS == 4) {
    const GroupParams g = grp[gv];
#pragma unroll
    for (int k = 0; k < kTileTokens; ++k) {
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t qa, qb;
        quantize_pair(w[e], g, L, qa, qb);
        col[2 * e] += qa << (BITS * k);
        col[2 * e + 1] += qb << (BITS * k);
      }
    }
  } else {
    // tokens 2a, 2a + 1 of channels 2e, 2e + 1 -> one word of four byte codes, then per channel
    // the bytes of tokens 0..3 and 4..7 -> two 8-bit fields
    const Thresh2 t = thr[gv];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t A[4];
#pragma unroll
      for (int a2 = 0; a2 < 4; ++a2) {
        const uint32_t w0 = comp4(x[2 * a2], e), w1 = comp4(x[2 * a2 + 1], e);
        A[a2] = __byte_perm(codes2_h2(w0, t), codes2_h2(w1, t), 0x6240);
      }
      col[2 * e] = gather4x2(__byte_perm(A[0], A[1], 0x5410)) | (gather4x2(__byte_perm(A[2], A[3], 0x5410)) << 8);
      col[2 * e + 1] = gather4x2(__byte_perm(A[0], A[1], 0x7632)) | (gather4x2(__byte_perm(A[2], A[3], 0x7632)) << 8);
    }
  }
  if constexpr (BITS == 4) {  // V word (tg, 8 c + e) holds exactly the tile's 8 tokens
    uint4* dst = reinterpret_cast<uint4*>(codes + tg * kHeadDim + 8 * c);
    dst[0] = make_uint4(col[0], col[1], col[2], col[3]);
    dst[1] = make_uint4(col[4], col[5], col[6], col[7]);
  } else {  // V word (tg / 2, 8 c + e): the even token group in bits 0..15, the odd one in 16..31
    const bool odd = tg & 1;
    uint32_t word[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // the even token group stores channels 0..3, the odd one 4..7
      const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? col[e] : col[4 + e], 16);
      word[e] = odd ? (other | (col[4 + e] << 16)) : (col[e] | (other << 16));
    }
    *reinterpret_cast<uint4*>(codes + (tg >> 1) * kHeadDim + 8 * c + (odd ? 4 : 0)) =
        make_uint4(word[0], word[1], word[2], word[3]);
  }
}

}  // namespace
}  // namespace kivi
