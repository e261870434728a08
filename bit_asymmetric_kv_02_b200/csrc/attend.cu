// Attention of one query token per sequence over quantized blocks of R tokens and fp16 residual rows,
// in pages or contiguous, with a sliding window and sinks.
//
//   out = softmax(scale q [D(Kq); Kres]^T) [D(Vq); Vres],  D(x^) = s x^ + z
//
// Split.  Each (row, KV head) is a run of 8 KB units: UT tokens of codes (128 at 2 bits, 64 at 4 bits:
// 4 KB of K, 4 KB of V) that hold a visible token, then 16 residual rows a unit.  All units of all rows,
// whose lengths differ, form one sequence, cut into one contiguous range per warp, so the load is even
// whatever the lengths; every CTA finds the ranges itself from a prefix sum of the rows' unit counts.
// A head that several warps share is joined by the warp that arrives last (its ticket), over the parts
// in their order: results do not depend on the order of arrival, and no warp waits for another.
// K and V halves arrive in shared memory by bulk copies, the next unit's K behind this unit's K.
//
// Products.  Both run on the tensor cores in fp16 with fp32 sums (mma m16n8k16), codes as the A operand:
// a masked code word IS a pair of fp16 subnormals, (w & 0x0003 << 2 j) = code 4^j 2^-24, exact, so an
// operand register of two codes costs one AND; the 4^-j goes into the B operand.  Codes at bits 10..15
// of a half are shifted down first.  The eight B columns hold four queries, each as two columns: the
// value rounded to fp16 and the rest, so operands carry 22 bits and nothing is lost to fp16:
//   K: B = q_c s_g(c) 2^x (s changes with every block: one multiply and one fused multiply-add a pair);
//      the constant sum_g z_g sum_c q_c is added in fp32.
//   V: B = p_t s_g(t) 2^y; sum_t p_t z_g(t) is one scalar per query.
// The column pair of a query sits in one lane, whose two sums are added there.  x and y are powers of
// two from the largest |q|, s of the block and s seen so far, which keep the operands inside fp16.
// Five to eight queries per KV head take two column blocks over the same A operands; more take passes.
// The tokens of a K tile are ordered so that a lane's logits are the pairs its P operand needs.
#include <cstdint>

#include "common.cuh"
#include "paged.h"

namespace kivi {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kResTokens = kAttendResTokens;      // tokens per residual unit
constexpr int kHalfBytes = 4096;                  // the K or the V part of a unit
constexpr int kKRow = 272;                        // a residual K row in shared memory (ldmatrix without conflicts)
constexpr int kVPiece = 1024, kVPieceStride = 1040;  // V word rows 2 t and 2 t + 1, four bank groups for t = 0..3
constexpr int kQRow = 272;                        // a raw query row in shared memory
constexpr int kPart = 132;                        // floats of a partial: m, l, Z, pad, o[128]
constexpr int kMaxCtas = 160;
constexpr uint64_t kWaitNs = 2000000000ull;       // bound of each wait for a copy
constexpr float kNoMax = -1e38f;                  // running maximum of no token: finite, so that exp2 of it minus itself is 1

#ifndef KIVI_ATTEND_WARPS
#define KIVI_ATTEND_WARPS 12
#endif
template <int NB>
__host__ __device__ constexpr int attend_warps() {
  return NB == 1 ? KIVI_ATTEND_WARPS : 8;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The codes of a word as pairs (j, j + P / 2) of fp16 subnormals: code 4^e(j) 2^-24 (16^e at 4 bits).
template <int BITS>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&a)[16 / BITS]) {
  if constexpr (BITS == 2) {
#pragma unroll
    for (int j = 0; j < 5; ++j) a[j] = w & (0x00030003u << (2 * j));
    const uint32_t w2 = w >> 10;
#pragma unroll
    for (int j = 5; j < 8; ++j) a[j] = w2 & (0x00030003u << (2 * (j - 5)));
  } else {
    const uint32_t w2 = w >> 8;
    a[0] = w & 0x000F000Fu;
    a[1] = w & 0x00F000F0u;
    a[2] = w2 & 0x000F000Fu;
    a[3] = w2 & 0x00F000F0u;
  }
}
// log2 of the factor code_pairs leaves on pair j.
template <int BITS>
__device__ __forceinline__ constexpr int pair_shift(int j) {
  return BITS == 2 ? 2 * (j < 5 ? j : j - 5) : 4 * (j & 1);
}

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

// The units of a row that hold a visible token: of the quantized ones the first q_sink and then those
// from q_sink + q_gap on (q_units in all), of the residual ones likewise.
struct Units {
  int q_sink, q_gap, q_units, r_sink, r_gap, total;
};
template <int UT>
__device__ __forceinline__ Units units_of(const Span& s) {
  Units u;
  const int nq = s.quant / UT;
  u.q_sink = min(nq, (s.sink_end + UT - 1) / UT);
  const int q0 = max(u.q_sink, min(nq, s.start / UT));
  u.q_gap = q0 - u.q_sink;
  u.q_units = nq - u.q_gap;
  const int nr = (s.len - s.quant + kResTokens - 1) / kResTokens;
  u.r_sink = min(nr, (max(0, s.sink_end - s.quant) + kResTokens - 1) / kResTokens);
  const int r0 = max(u.r_sink, min(nr, max(0, s.start - s.quant) / kResTokens));
  u.r_gap = r0 - u.r_sink;
  u.total = max(1, u.q_units + nr - u.r_gap);  // a row without tokens has one unit, which finds nothing
  return u;
}

// Row of q and out that sequence b takes, or -1.
__device__ __forceinline__ int q_row(const AttendArgs& a, int b, bool* bad) {
  int row = b;
  if (a.cu_tokens != nullptr) {
    const int next = __ldg(a.cu_tokens + b + 1);
    if (next == __ldg(a.cu_tokens + b)) return -1;
    row = next - 1;
  }
  if (row < 0 || row >= a.q_rows) {
    *bad = true;
    return -1;
  }
  return row;
}

template <int BITS, int NB>
struct __align__(128) WarpSmem {
  uint8_t k[kResTokens * kKRow];
  uint8_t v[4 * kVPieceStride];
  uint4 p[NB][BITS == 2 ? 128 : 64];  // P operands: column, code pair and word rows (p_slot)
  uint8_t q[NB][4 * kQRow];           // the head's raw queries
  uint64_t bar[2];
};

template <int BITS, int NB>
struct Attender {
  static constexpr int P = 32 / BITS;               // codes per word
  static constexpr int HP = P / 2;                  // code pairs per word
  static constexpr int UT = attend_unit_tokens(BITS);  // tokens per quantized unit
  static constexpr int PT = UT / 4;                 // tokens of two V word rows
  static constexpr int MT = UT / 16;                // K tiles per unit
  static constexpr int KW = kHeadDim / P / 4;       // K words per lane and token
  static constexpr int NQ = 4 * NB;                 // queries a warp holds
  using Smem = WarpSmem<BITS, NB>;

  const AttendArgs& a;
  Smem& S;
  const int* cum;  // [rows + 1] units per head before each row
  const int lane, g, t;
  const int he_count;  // (KV head, pass) pairs per row
  long long worker, workers, total;

  // a unit: where its halves are, and which of its tokens are visible
  struct Unit {
    long long off;           // bytes from the start of the K and V arrays
    long long ks, vs;        // first (s, z) of the block
    int tok0, start, sink_end, len;
    bool ok, res, full;
  };
  // the position of the unit that is fetched next
  int seq, he, local;
  Units un;
  Span sp;

  // state of the head in hand: lane (g, t) is query t (of each column block) and channels 16 g .. 16 g + 15
  uint32_t qh[NB][16];  // B-operand share of lane (column g, t): channels 32 t .. 32 t + 31 of query g / 2, scaled
  float m[NB], l[NB], Z[NB], o[NB][8][4];
  float qs[NB][4];   // scale * log2 e * sum of q over channels 32 i .. 32 i + 31
  int qe[NB];        // exponent of the largest |q|
  int eref;          // exponent field of the largest V scale so far: o carries 2^(28 - eref - 24)
  uint32_t kphase, vphase;

  __device__ Attender(const AttendArgs& args, Smem& smem, const int* c, int ln)
      : a(args), S(smem), cum(c), lane(ln), g(ln >> 2), t(ln & 3), he_count(args.heads * args.passes), kphase(0), vphase(0) {}

  // ---- units ---------------------------------------------------------------------------------------
  __device__ void set_seq(int i) {
    seq = i;
    bool bad;
    sp = span_of(a, i, &bad);
    un = units_of<UT>(sp);
  }
  __device__ void seek(long long f) {
    const int want = static_cast<int>(f / he_count);
    int lo = 0, hi = a.rows;  // cum[lo] <= want < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= want)
        lo = mid;
      else
        hi = mid;
    }
    set_seq(lo);
    const long long rem = f - static_cast<long long>(cum[lo]) * he_count;
    he = static_cast<int>(rem / un.total);
    local = static_cast<int>(rem - static_cast<long long>(he) * un.total);
  }
  __device__ void advance() {
    if (++local < un.total) return;
    local = 0;
    if (++he < he_count) return;
    he = 0;
    int i = seq + 1;
    while (i < a.rows && cum[i + 1] == cum[i]) ++i;
    if (i < a.rows) set_seq(i);
  }
  __device__ Unit fetch() const {
    Unit u;
    const int h = a.passes == 1 ? he : he / a.passes;
    u.len = sp.len;
    u.start = sp.start;
    u.sink_end = sp.sink_end;
    u.res = local >= un.q_units;
    u.ok = true;
    u.ks = u.vs = 0;
    int n;
    if (!u.res) {
      int x = local;
      if (x >= un.q_sink) x += un.q_gap;
      u.tok0 = x * UT;
      n = UT;
      const int j = u.tok0 >> a.lg_r, in = u.tok0 & ((1 << a.lg_r) - 1);
      long long blk;
      if (a.block_table != nullptr) {
        const int page = __ldg(a.block_table + static_cast<size_t>(seq) * a.max_blocks + j);  // j < max_blocks: span_of
        u.ok = page >= 0 && page < a.num_pages;
        blk = static_cast<long long>(u.ok ? page : 0) * a.heads + h;
        if (!u.ok && lane == 0) report_status(a.status, KIVI_ERR_INTERNAL);
      } else {
        blk = (static_cast<long long>(seq) * a.heads + h) * a.blocks_per_head + j;
      }
      u.off = ((blk << a.lg_r) + in) * (kHeadDim * BITS / 8);
      u.ks = blk * (kHeadDim >> a.lg_gk) + ((32 * t) >> a.lg_gk);
      u.vs = (blk << a.lg_r >> a.lg_gv) + ((in + PT * t) >> a.lg_gv);
    } else {
      int x = local - un.q_units;
      if (x >= un.r_sink) x += un.r_gap;
      u.tok0 = sp.quant + x * kResTokens;
      n = kResTokens;
      u.ok = u.tok0 < sp.len;
      u.off = (((static_cast<long long>(seq) * a.heads + h) << a.lg_r) + x * kResTokens) * (kHeadDim * 2);
    }
    u.full = u.tok0 + n <= u.sink_end || (u.tok0 >= u.start && u.tok0 + n <= u.len);
    return u;
  }
  __device__ void issue_k(const Unit& u) {
    if (!u.ok) return;
    if (lane == 0) mbar_arrive_expect_tx(&S.bar[0], kHalfBytes);
    __syncwarp();
    if (!u.res) {
      if (lane == 0) bulk_g2s(S.k, reinterpret_cast<const char*>(a.k_codes) + u.off, kHalfBytes, &S.bar[0]);
    } else if (lane < kResTokens) {
      bulk_g2s(S.k + lane * kKRow, reinterpret_cast<const char*>(a.k_res) + u.off + lane * 256, 256, &S.bar[0]);
    }
  }
  __device__ void issue_v(const Unit& u) {
    if (!u.ok) return;
    if (lane == 0) mbar_arrive_expect_tx(&S.bar[1], kHalfBytes);
    __syncwarp();
    const char* src = u.res ? reinterpret_cast<const char*>(a.v_res) : reinterpret_cast<const char*>(a.v_codes);
    if (lane < 4) bulk_g2s(S.v + lane * kVPieceStride, src + u.off + lane * kVPiece, kVPiece, &S.bar[1]);
  }
  // (s, z) of this lane's piece: K channels 32 t .. 32 t + 31 and V tokens PT t .. PT t + PT - 1
  __device__ void load_pairs(const Unit& u, uint32_t& kp, uint32_t& vp) const {
    kp = vp = 0;
    if (!u.ok || u.res) return;
    kp = static_cast<uint32_t>(__ldg(a.k_scale + u.ks)) | (static_cast<uint32_t>(__ldg(a.k_zero + u.ks)) << 16);
    vp = static_cast<uint32_t>(__ldg(a.v_scale + u.vs)) | (static_cast<uint32_t>(__ldg(a.v_zero + u.vs)) << 16);
  }
  __device__ static bool seen(const Unit& u, int tok) { return tok < u.len && (tok < u.sink_end || tok >= u.start); }

  // ---- the head's queries ----------------------------------------------------------------------------
  __device__ void start_head() {
    const int h = he / a.passes, pass = he - h * a.passes;
    bool bad = false;
    const int row = q_row(a, seq, &bad);
    const int q0 = pass * a.per_pass, nq = min(a.per_pass, a.gqa - q0);
    const uint16_t* base = a.q + (static_cast<size_t>(row) * a.heads * a.gqa + static_cast<size_t>(h) * a.gqa + q0) * kHeadDim;
    __syncwarp();  // the previous head's raw queries are no longer read
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int qi = 4 * b + (g >> 1);
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = qi < nq ? __ldg(reinterpret_cast<const uint4*>(base + static_cast<size_t>(qi) * kHeadDim + 32 * t) + i)
                       : make_uint4(0, 0, 0, 0);
      if ((g & 1) == 0) {
        uint4* dst = reinterpret_cast<uint4*>(S.q[b] + (g >> 1) * kQRow + 64 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = v[i];
      }
      float f[32], big = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = unpack_h2(w[j]);
          f[8 * i + 2 * j] = x.x;
          f[8 * i + 2 * j + 1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        big = fmaxf(big, fabsf(f[i]));
        sum += f[i];
      }
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
      const int e = big > 0.f ? (__float_as_int(big) >> 23) - 127 : 0;  // -24 .. 16
#pragma unroll
      for (int x = 0; x < KW; ++x)
#pragma unroll
        for (int j = 0; j < HP; ++j) {
          const float sc = pow2i(6 - e - pair_shift<BITS>(j));
          qh[b][x * HP + j] = pack_h2(f[x * P + j] * sc, f[x * P + j + HP] * sc);
        }
      qe[b] = __shfl_sync(kFull, e, 8 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[b][i] = a.qscale * __shfl_sync(kFull, sum, 8 * t + i);
      m[b] = kNoMax;
      l[b] = Z[b] = 0.f;
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[b][v8][i] = 0.f;
    }
    eref = 1;
    __syncwarp();
  }

  // o, l and Z move to a new running maximum and V scale exponent.
  __device__ __forceinline__ void raise(int b, float mu, float escale) {
    float mx = fmaxf(mu, __shfl_xor_sync(kFull, mu, 4));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
    const float mn = fmaxf(m[b], mx), al = ex2(m[b] - mn), ao = al * escale;
    m[b] = mn;
    l[b] *= al;
    Z[b] *= al;
#pragma unroll
    for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[b][v8][i] *= ao;
  }

  // Slot of P operand vector (column n, code pair jl of word rows of lane tt): conflict-free for the
  // lanes that write one (jl and tt fixed by g, columns 2 t + lo) and those that read it (n = g, tt = t).
  __device__ static __forceinline__ int p_slot(int n, int jl, int tt) {
    return n * 16 + ((jl * 4 + tt) ^ ((n >> 1) | ((n & 1) << 2)));
  }

  // ---- K half of a quantized unit: logits, softmax, P operands ------------------------------------------
  // Tile i = (tb, x, jj) (2 bits) or (tb, x) holds on rows g and g + 8 the tokens of pair j = 4 jj + g % 4 (g % 4)
  // of word row 2 tt + x, tt = 2 (g / 4) + tb: what lane tt of the V product needs as one operand register.
  __device__ void quant_k(const Unit& u, uint32_t kp, uint32_t vp) {
    const int jl = g & 3, tt0 = (g >> 2) * 2;
    if (!u.full) {  // V pieces that are hidden whole have no say (their s and z may be anything)
      const int p0 = u.tok0 + PT * t;
      if (p0 >= u.sink_end && p0 + PT <= u.start) vp = 0;
    }
    const unsigned ksm = __reduce_max_sync(kFull, kp & 0xFFFFu), vsm = __reduce_max_sync(kFull, vp & 0xFFFFu);
    const int ek = max(1, static_cast<int>(ksm >> 10)), ev = max(1, static_cast<int>(vsm >> 10));
    const __half2 sh = __float2half2_rn(h2f(static_cast<uint16_t>(kp)) * pow2i(22 - ek));
    const __half2 shl = (g & 1) ? sh : __float2half2_rn(0.f);
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = h2f(static_cast<uint16_t>(__shfl_sync(kFull, kp, i) >> 16));
    uint32_t kb[NB][16];
    float inv[NB], cst[NB], lg[NB][MT][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __half2 q2 = as_h2(qh[b][i]);
        kb[b][i] = as_u32(__hfma2(q2, sh, __hneg2(__hmul2(q2, shl))));  // even columns: q s rounded; odd: the rest
      }
      inv[b] = a.qscale * pow2i(qe[b] + ek - 4);
      cst[b] = fmaf(z[3], qs[b][3], fmaf(z[2], qs[b][2], fmaf(z[1], qs[b][1], z[0] * qs[b][0])));
    }
    const uint8_t* kt = S.k + ((g >> 2) * (UT / 2) + jl) * (16 * BITS) + 4 * KW * t;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int off = BITS == 2 ? (i >> 2) * 1024 + ((i >> 1) & 1) * 512 + (i & 1) * 128 : (i >> 1) * 1024 + (i & 1) * 512;
      uint32_t wg[KW], wh[KW];
      if constexpr (BITS == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(kt + off), y = *reinterpret_cast<const uint2*>(kt + off + 256);
        wg[0] = x.x, wg[1] = x.y, wh[0] = y.x, wh[1] = y.y;
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(kt + off), y = *reinterpret_cast<const uint4*>(kt + off + 256);
        wg[0] = x.x, wg[1] = x.y, wg[2] = x.z, wg[3] = x.w, wh[0] = y.x, wh[1] = y.y, wh[2] = y.z, wh[3] = y.w;
      }
      float c[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b) c[b][0] = c[b][1] = c[b][2] = c[b][3] = 0.f;
#pragma unroll
      for (int x = 0; x < KW; ++x) {
        uint32_t ag[HP], ah[HP];
        code_pairs<BITS>(wg[x], ag);
        code_pairs<BITS>(wh[x], ah);
#pragma unroll
        for (int j = 0; j < HP; j += 2)
#pragma unroll
          for (int b = 0; b < NB; ++b) mma16(c[b], ag[j], ah[j], ag[j + 1], ah[j + 1], kb[b][x * HP + j], kb[b][x * HP + j + 1]);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        lg[b][i][0] = fmaf(c[b][0] + c[b][1], inv[b], cst[b]);
        lg[b][i][1] = fmaf(c[b][2] + c[b][3], inv[b], cst[b]);
      }
    }
    if (!u.full) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int tok = BITS == 2 ? u.tok0 + 32 * (tt0 + (i >> 2)) + 16 * ((i >> 1) & 1) + 4 * (i & 1) + jl
                                  : u.tok0 + 16 * (tt0 + (i >> 1)) + 8 * (i & 1) + jl;
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (!seen(u, tok + HP * y))
#pragma unroll
            for (int b = 0; b < NB; ++b) lg[b][i][y] = -INFINITY;
      }
    }
    float mu[NB];
    bool up = ev > eref;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      mu[b] = lg[b][0][0];
#pragma unroll
      for (int i = 0; i < MT; ++i) mu[b] = fmaxf(mu[b], fmaxf(lg[b][i][0], lg[b][i][1]));
      up = up || mu[b] > m[b];
    }
    if (__any_sync(kFull, up)) {
      const float escale = pow2i(min(0, eref - ev));
      eref = max(eref, ev);
#pragma unroll
      for (int b = 0; b < NB; ++b) raise(b, mu[b], escale);
    }
    const float kscale = pow2i(28 - eref);
    uint32_t vq[2] = {__shfl_sync(kFull, vp, tt0), __shfl_sync(kFull, vp, tt0 + 1)};
    constexpr int JJ = BITS == 2 ? 2 : 1;
    float fac[2][JJ];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb) {
      const float s = h2f(static_cast<uint16_t>(vq[tb])) * kscale;
      if constexpr (BITS == 2) {
        fac[tb][0] = s * pow2i(-2 * jl);
        fac[tb][1] = s * (jl == 0 ? 0x1p-8f : pow2i(2 - 2 * jl));
      } else {
        fac[tb][0] = (jl & 1) ? s * 0x1p-4f : s;
      }
    }
    constexpr int HALF = MT / 2;  // tiles of one tb
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        uint32_t hi[HALF], lo[HALF];
        float ps = 0.f;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
          const float p0 = ex2(lg[b][tb * HALF + i][0] - m[b]), p1 = ex2(lg[b][tb * HALF + i][1] - m[b]);
          ps += p0 + p1;
          const float f = fac[tb][JJ == 2 ? i & 1 : 0], x0 = p0 * f, x1 = p1 * f;
          hi[i] = pack_h2(x0, x1);
          const float2 r = unpack_h2(hi[i]);
          lo[i] = pack_h2(x0 - r.x, x1 - r.y);
        }
        l[b] += ps;
        Z[b] = fmaf(ps, h2f(static_cast<uint16_t>(vq[tb] >> 16)), Z[b]);
        if constexpr (BITS == 2) {
          S.p[b][p_slot(2 * t, jl, tt0 + tb)] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          S.p[b][p_slot(2 * t + 1, jl, tt0 + tb)] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        } else {
          uint2* p2 = reinterpret_cast<uint2*>(S.p[b]);
          p2[p_slot(2 * t, jl, tt0 + tb)] = make_uint2(hi[0], hi[1]);
          p2[p_slot(2 * t + 1, jl, tt0 + tb)] = make_uint2(lo[0], lo[1]);
        }
      }
    }
  }

  // ---- V half of a quantized unit: tile v8 holds channels 16 g + 2 v8 (row g) and 16 g + 2 v8 + 1 (row g + 8) ----
  __device__ void quant_v() {
    uint32_t pb[NB][2][HP];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int jl = 0; jl < 4; ++jl) {
        if constexpr (BITS == 2) {
          const uint4 x = S.p[b][p_slot(g, jl, t)];
          pb[b][0][jl] = x.x, pb[b][0][4 + jl] = x.y, pb[b][1][jl] = x.z, pb[b][1][4 + jl] = x.w;
        } else {
          const uint2 x = reinterpret_cast<const uint2*>(S.p[b])[p_slot(g, jl, t)];
          pb[b][0][jl] = x.x, pb[b][1][jl] = x.y;
        }
      }
    const uint8_t* vt = S.v + t * kVPieceStride + 64 * g;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(vt + x * 512 + 16 * i);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t ag[HP], ah[HP];
          code_pairs<BITS>(w[2 * e], ag);
          code_pairs<BITS>(w[2 * e + 1], ah);
#pragma unroll
          for (int j = 0; j < HP; j += 2)
#pragma unroll
            for (int b = 0; b < NB; ++b)
              mma16(o[b][2 * i + e], ag[j], ah[j], ag[j + 1], ah[j + 1], pb[b][x][j], pb[b][x][j + 1]);
        }
      }
  }

  // ---- residual units: K on the tensor cores with the raw queries, V with fp32 multiply-adds ------------
  __device__ void res_k(const Unit& u, float (&p)[NB][2]) {
    float c[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) c[b][0] = c[b][1] = c[b][2] = c[b][3] = 0.f;
    const uint32_t row = smem_u32(S.k) + (lane & 15) * kKRow + (lane >> 4) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t x[4];
      ldmatrix4(x, row + 32 * i);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(S.q[b] + (g >> 1) * kQRow) + 8 * i + t;
        const uint32_t b0 = (g & 1) ? 0u : q[0], b1 = (g & 1) ? 0u : q[4];
        mma16(c[b], x[0], x[1], x[2], x[3], b0, b1);
      }
    }
    const bool s0 = seen(u, u.tok0 + g), s1 = seen(u, u.tok0 + g + 8);
    bool up = false;
    float mu[NB], lg[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      lg[b][0] = s0 ? (c[b][0] + c[b][1]) * a.qscale : -INFINITY;
      lg[b][1] = s1 ? (c[b][2] + c[b][3]) * a.qscale : -INFINITY;
      mu[b] = fmaxf(lg[b][0], lg[b][1]);
      up = up || mu[b] > m[b];
    }
    if (__any_sync(kFull, up)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) raise(b, mu[b], 1.f);
    }
    const float oscale = pow2i(4 - eref);  // o carries 2^(28 - eref - 24)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float p0 = ex2(lg[b][0] - m[b]), p1 = ex2(lg[b][1] - m[b]);
      l[b] += p0 + p1;
      p[b][0] = p0 * oscale;
      p[b][1] = p1 * oscale;
    }
  }
  __device__ void res_v(const Unit& u, const float (&p)[NB][2]) {
#pragma unroll 1
    for (int j = 0; j < kResTokens; ++j) {
      if (!seen(u, u.tok0 + j)) continue;  // the same for every lane; rows that are hidden may hold anything
      const uint4* src = reinterpret_cast<const uint4*>(S.v + (j >> 2) * kVPieceStride + (j & 3) * 256 + 32 * g);
      const uint4 x = src[0], y = src[1];
      const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float pj = __shfl_sync(kFull, j < 8 ? p[b][0] : p[b][1], (j & 7) * 4 + t);
#pragma unroll
        for (int v8 = 0; v8 < 8; ++v8) {
          const float2 f = unpack_h2(w[v8]);
          o[b][v8][0] = fmaf(pj, f.x, o[b][v8][0]);
          o[b][v8][2] = fmaf(pj, f.y, o[b][v8][2]);
        }
      }
    }
  }

  // ---- the end of a head's segment -----------------------------------------------------------------------
  // Lane (g, t): o of query t (each column block), channels 16 g .. 16 g + 15.
  __device__ void finish(bool whole, int slot) {
    const int h = he_now / a.passes, pass = he_now - h * a.passes;
    const int q0 = pass * a.per_pass, nq = min(a.per_pass, a.gqa - q0);
    const float back = pow2i(eref - 4);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float ls = l[b], zs = Z[b];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        ls += __shfl_xor_sync(kFull, ls, off);
        zs += __shfl_xor_sync(kFull, zs, off);
      }
      const int qi = 4 * b + t;
      if (qi >= nq) continue;
      float f[16];
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8) {
        f[2 * v8] = (o[b][v8][0] + o[b][v8][1]) * back;
        f[2 * v8 + 1] = (o[b][v8][2] + o[b][v8][3]) * back;
      }
      if (whole) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_h2((f[2 * i] + zs) * inv, (f[2 * i + 1] + zs) * inv);
        uint4* dst = reinterpret_cast<uint4*>(
            a.out + (static_cast<size_t>(row_now) * a.heads * a.gqa + static_cast<size_t>(h) * a.gqa + q0 + qi) * kHeadDim + 16 * g);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        float* dst = a.partials + ((worker * 2 + slot) * NQ + qi) * kPart;
        if (g == 0) *reinterpret_cast<float4*>(dst) = make_float4(m[b], ls, zs, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(dst + 4 + 16 * g + 4 * i) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
    }
  }

  // Worker whose range holds unit f: ranges start at floor(total w / workers).
  __device__ __forceinline__ long long worker_of(long long f) const { return ((f + 1) * workers + total - 1) / total - 1; }

  // The workers that hold a part of a head left one partial each: the first of them in its slot 1
  // unless its range starts with the head, the others in their slot 0.
  __device__ void merge(int s, int e, long long f0, int units) {
    const long long w0 = worker_of(f0), w1 = worker_of(f0 + units - 1);
    const int parts = static_cast<int>(w1 - w0 + 1);
    const int slot0 = total * w0 / workers >= f0 ? 0 : 1;
    const int h = e / a.passes, pass = e - h * a.passes;
    const int q0 = pass * a.per_pass, nq = min(a.per_pass, a.gqa - q0);
    bool bad = false;
    const int row = q_row(a, s, &bad);
#pragma unroll 1
    for (int qi = 0; qi < nq; ++qi) {
      auto part = [&](int k) { return a.partials + (((w0 + k) * 2 + (k == 0 ? slot0 : 0)) * NQ + qi) * kPart; };
      float mx = kNoMax;
      for (int k = lane; k < parts; k += 32) mx = fmaxf(mx, __ldcg(part(k)));
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
      float ls = 0.f, zs = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k0 = 0; k0 < parts; k0 += 32) {
        float w = 0.f;
        if (k0 + lane < parts) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(part(k0 + lane)));
          w = ex2(x.x - mx);
          ls = fmaf(w, x.y, ls);
          zs = fmaf(w, x.z, zs);
        }
        const int n = min(32, parts - k0);
        for (int i = 0; i < n; i += 16) {
          float4 v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = i + j < n ? __ldcg(reinterpret_cast<const float4*>(part(k0 + i + j) + 4) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float wj = __shfl_sync(kFull, w, (i + j) & 31);
            acc[0] = fmaf(wj, v[j].x, acc[0]);
            acc[1] = fmaf(wj, v[j].y, acc[1]);
            acc[2] = fmaf(wj, v[j].z, acc[2]);
            acc[3] = fmaf(wj, v[j].w, acc[3]);
          }
        }
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        ls += __shfl_xor_sync(kFull, ls, off);
        zs += __shfl_xor_sync(kFull, zs, off);
      }
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(row) * a.heads * a.gqa + static_cast<size_t>(h) * a.gqa + q0 + qi) * kHeadDim +
                                4 * lane) =
          make_uint2(pack_h2((acc[0] + zs) * inv, (acc[1] + zs) * inv), pack_h2((acc[2] + zs) * inv, (acc[3] + zs) * inv));
    }
    if (lane == 0) a.tickets[static_cast<size_t>(s) * he_count + e] = 0;
  }

  __device__ bool wait(int which, uint32_t& phase) {
    const bool ok = __all_sync(kFull, mbar_wait_bounded(&S.bar[which], phase, kWaitNs));
    phase ^= 1;
    return ok;
  }

  int he_now, row_now;

  __device__ void run(long long w, long long nw, long long all) {
    worker = w;
    workers = nw;
    total = all;
    const long long f0 = total * w / workers, f1 = total * (w + 1) / workers;
    if (lane == 0) {
      mbar_init(&S.bar[0], 1);
      mbar_init(&S.bar[1], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    seek(f0);
    Unit nx = fetch();
    issue_k(nx);
    issue_v(nx);
    uint32_t kp, vp;
    load_pairs(nx, kp, vp);
    struct Head {
      int seq, he, units;
      long long f0;
    } pend[2];
    int npend = 0;
    long long left = f1 - f0;
    bool first = true;
    while (left > 0) {
      const int s = seq, e = he, l0 = local, units = un.total;
      const int count = static_cast<int>(min(left, static_cast<long long>(units - local)));
      bool bad = false;
      he_now = he;
      row_now = q_row(a, seq, &bad);
      start_head();
      for (int i = 0; i < count; ++i) {
        const Unit cu = nx;
        const uint32_t ckp = kp, cvp = vp;
        const bool more = left - i > 1;
        if (more) {
          advance();
          nx = fetch();
        }
        float p[NB][2];
        if (cu.ok) {
          if (!wait(0, kphase)) {
            if (lane == 0) report_status(a.status, KIVI_ERR_DEVICE_TIMEOUT);
            (void)mbar_wait_bounded(&S.bar[1], vphase, kWaitNs);  // no copy in flight when the warp ends
            return;
          }
          if (!cu.res)
            quant_k(cu, ckp, cvp);
          else
            res_k(cu, p);
        }
        __syncwarp();  // the K half has been read, and the P operands are written
        if (more) {
          issue_k(nx);
          load_pairs(nx, kp, vp);
        }
        if (cu.ok) {
          if (!wait(1, vphase)) {
            if (lane == 0) report_status(a.status, KIVI_ERR_DEVICE_TIMEOUT);
            if (more && nx.ok) (void)mbar_wait_bounded(&S.bar[0], kphase, kWaitNs);
            return;
          }
          if (!cu.res)
            quant_v();
          else
            res_v(cu, p);
        }
        __syncwarp();
        if (more) issue_v(nx);
      }
      const bool whole = count == units;
      finish(whole, first ? 0 : 1);
      if (!whole) {
        pend[npend].seq = s;
        pend[npend].he = e;
        pend[npend].units = units;
        pend[npend].f0 = f1 - left - l0;
        ++npend;
      }
      left -= count;
      first = false;
    }
    if (npend == 0) return;
    // one fence publishes this warp's partials before its tickets; the last part of a head joins it
    __threadfence();
    __syncwarp();
    int last = 0;
    if (lane == 0) {
      for (int i = 0; i < npend; ++i) {
        const int others = static_cast<int>(worker_of(pend[i].f0 + pend[i].units - 1) - worker_of(pend[i].f0));
        if (atomicAdd(a.tickets + static_cast<size_t>(pend[i].seq) * he_count + pend[i].he, 1) == others) last |= 1 << i;
      }
      if (last) __threadfence();
    }
    last = __shfl_sync(kFull, last, 0);
    if (!last) return;
    __threadfence();
#pragma unroll 1
    for (int i = 0; i < npend; ++i)
      if ((last >> i) & 1) merge(pend[i].seq, pend[i].he, pend[i].f0, pend[i].units);
  }
};

template <int BITS, int NB>
__global__ void __launch_bounds__(attend_warps<NB>() * 32, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int W = attend_warps<NB>(), T = W * 32;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Smem = WarpSmem<BITS, NB>;
  int* cum = reinterpret_cast<int*>(smem_raw + W * sizeof(Smem));
  __shared__ int warp_sum[W];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // units per head of every row, and their prefix sums (rows below 8193, sums below 2^31)
  const int per = (a.rows + T - 1) / T, r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
  int mine = 0;
  for (int i = r0; i < r1; ++i) {
    bool bad = false, bad_row = false;
    const int row = q_row(a, i, &bad_row);
    const int n = row < 0 ? 0 : units_of<Attender<BITS, NB>::UT>(span_of(a, i, &bad)).total;
    if ((bad || bad_row) && blockIdx.x == 0) report_status(a.status, KIVI_ERR_INTERNAL);
    cum[i] = n;
    mine += n;
  }
  int x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(kFull, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = x - mine;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  for (int i = r0; i < r1; ++i) {
    const int n = cum[i];
    cum[i] = before;
    before += n;
  }
  if (r0 < a.rows && r1 == a.rows) cum[a.rows] = before;
  __syncthreads();
  const long long total = static_cast<long long>(cum[a.rows]) * a.heads * a.passes;
  const long long workers = min(total, static_cast<long long>(gridDim.x) * W);
  // neighbouring workers on different SMs: few units spread over the GPU
  const long long worker = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  if (worker >= workers) return;
  Attender<BITS, NB> d(a, reinterpret_cast<Smem*>(smem_raw)[warp], cum, lane);
  d.run(worker, workers, total);
}

template <int BITS, int NB>
cudaError_t launch(const AttendArgs& a, int ctas, cudaStream_t stream) {
  const size_t smem = attend_warps<NB>() * sizeof(WarpSmem<BITS, NB>) + (static_cast<size_t>(a.rows) + 1) * sizeof(int);
  static_assert(attend_warps<NB>() * sizeof(WarpSmem<BITS, NB>) + 8193 * 4 + 128 <= 232448, "a CTA holds 227 KB of shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(attend_kernel<BITS, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  attend_kernel<BITS, NB><<<ctas, attend_warps<NB>() * 32, smem, stream>>>(a);
  return cudaGetLastError();
}

struct Shape {
  int passes, per_pass, blocks;  // query passes per KV head, queries of a pass, column blocks of four queries
  long long workers;             // at most
};
Shape shape_of(long long rows, int heads, int gqa, long long max_units) {
  Shape s;
  s.passes = (gqa + 7) / 8;
  s.per_pass = (gqa + s.passes - 1) / s.passes;
  s.blocks = s.per_pass > 4 ? 2 : 1;
  const long long warps = static_cast<long long>(kMaxCtas) * (s.blocks == 1 ? attend_warps<1>() : attend_warps<2>());
  const long long heads_all = rows * heads * s.passes;
  s.workers = heads_all == 0 || max_units > warps / heads_all ? warps : heads_all * max_units;
  return s;
}
size_t ticket_bytes(long long rows, int heads, const Shape& s) {
  return (static_cast<size_t>(rows) * heads * s.passes * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

}  // namespace

size_t attend_workspace_bytes(long long rows, int heads, int gqa, long long max_units) {
  const Shape s = shape_of(rows, heads, gqa, max_units);
  const size_t part = static_cast<size_t>(s.workers) * 2 * 4 * s.blocks * kPart * sizeof(float);
  return ticket_bytes(rows, heads, s) + ((part + 255) & ~static_cast<size_t>(255));
}

cudaError_t launch_attend(AttendArgs a, int bits, long long max_units, void* workspace, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const Shape s = shape_of(a.max_rows, a.heads, a.gqa, max_units);
  a.passes = s.passes;
  a.per_pass = s.per_pass;
  a.tickets = static_cast<int32_t*>(workspace);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + ticket_bytes(a.max_rows, a.heads, s));
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int warps = s.blocks == 1 ? attend_warps<1>() : attend_warps<2>();
  long long ctas = sms < kMaxCtas ? sms : kMaxCtas;
  // a worker per warp at most: fewer CTAs than SMs only where fewer units can exist
  if (ctas * warps > s.workers) ctas = s.workers < ctas ? s.workers : ctas;
  if (bits == 2)
    return s.blocks == 1 ? launch<2, 1>(a, static_cast<int>(ctas), stream) : launch<2, 2>(a, static_cast<int>(ctas), stream);
  return s.blocks == 1 ? launch<4, 1>(a, static_cast<int>(ctas), stream) : launch<4, 2>(a, static_cast<int>(ctas), stream);
}

}  // namespace kivi
