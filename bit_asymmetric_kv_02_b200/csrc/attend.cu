// Attention of one query token per sequence over quantized blocks of R tokens and fp16 residual rows,
// in pages or contiguous, with a sliding window and sinks.
//
//   out = softmax(scale q [D(Kq); Kres]^T) [D(Vq); Vres],  D(x^) = s x^ + z
//
// Split.  Each (row, KV head) is a run of 8 KB units: UT tokens of codes (128 at 2 bits, 64 at 4 bits:
// 4 KB of K, 4 KB of V) that hold a visible token, then 16 residual rows a unit.  All units of all rows,
// whose lengths differ, form one sequence, cut into one contiguous range per warp, so the load is even
// whatever the lengths; every CTA finds the ranges itself from a prefix sum of the rows' unit counts.
// Heads that several warps share are joined in shared memory behind the CTA's last barrier, and across CTAs by the warp that
// arrives last at a ticket, over the parts in their order: results do not depend on the order of arrival, and no CTA waits for
// another.
// K and V halves arrive in shared memory by 16-byte asynchronous copies, the next unit's K behind this unit's K (bulk copies,
// of which a warp issues one at a time, cost 200 instructions a unit in loops over the pieces).
//
// Products.  Both run on the tensor cores in fp16 with fp32 sums (mma m16n8k16), codes as the A operand:
// a masked code word IS a pair of fp16 subnormals, code 2^(b - 24) at bit b of its half, exact, so an
// operand register of two codes costs one AND; what b leaves over goes into the B operand.  Codes at bits 0..3
// of a half are shifted up by 4 and those at 10..15 down by 6 first (2 bits): products of the smallest subnormals lose their
// last bits in the tensor cores' sums (16 x 8 x 4 queries up to 32768 tokens: error before the rounding 5.0e-5 of the output
// with codes at bits 0..9, 6.6e-6 with 4..9, in the same time).  The eight B columns hold four queries, each as two columns: the
// value rounded to fp16 and the rest, so operands carry 22 bits and nothing is lost to fp16:
//   K: B = q_c s_g(c) 2^x (s changes with every block: one multiply and one fused multiply-add a pair);
//      the constant sum_g z_g sum_c q_c is added in fp32.
//   V: B = p_t s_g(t) 2^y; sum_t p_t z_g(t) is one scalar per query.
// The column pair of a query sits in one lane, whose two sums are added there.  x and y are powers of
// two, x from the largest |q| and s of the block, y from the largest p_t s_g(t) of the unit, for each query: the operands stay
// inside fp16, and a group of large values that has no weight takes no bits from those that have.
// Five to eight queries per KV head take two column blocks over the same A operands; more take passes.
// The tokens of a K tile are ordered so that a lane's logits are the pairs its P operand needs.
// One query per KV head takes integer products of bytes instead (struct One).
//
// What bounds it.  Read-only streams reach about the copy bandwidth here (6.46 TB/s), 1.25 us for the 8 KB of
// every SM.  An SM issues an mma m16n8k16 every 2.0 clocks and a logic instruction for four warps every 2, and
// beside an mma four of the latter take 2.8: with 128 products and 640 masks and shifts per 8 KB at 2 bits, the
// instructions set the time for 2 to 4 queries (570 clocks per 8 KB, 47% of the copy bandwidth), and at
// 4 bits, with half of either, nearly so.  One query on bytes (192 masks, 64 products) comes to 75% to 85%.
//   64 rows of up to 8192 tokens x 32 heads, 2 bits:                177 us; 156 on other GPUs (859 MB)
//   4 rows of up to 32001 tokens x 32 heads, 4 bits:                 95 us (502 MB)
//   16 rows of up to 32768 tokens x 8 KV heads x 4 queries, 2 bits:  67 us (204 MB); 4 bits: 92 us (402 MB); 8 queries, 2 bits: 104 us
//   16 rows of up to 32768 tokens x 1 KV head x 8, 32 and 64 queries, 2 bits: 27, 60 and 102 us (a pass of 8 after the other)
// The rest is start and end: about 2 us until the ranges are known, 3.5 us for the first unit, 1.5 us to join heads in a CTA,
// 3 us and more across CTAs.
#include <cstdint>

#include "common.cuh"
#include "overlap.cuh"
#include "paged.h"

namespace kivi {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kResTokens = kAttendResTokens;      // tokens per residual unit
constexpr int kHalfBytes = 4096;                  // the K or the V part of a unit
constexpr int kRow = 272;                         // a residual row in shared memory (ldmatrix without conflicts)
constexpr int kVPieceStride = 1040;               // V word rows 2 t and 2 t + 1, four bank groups for t = 0..3
constexpr int kQRow = 272;                        // a raw query row in shared memory
constexpr int kPart = 132;                        // floats of a partial: m, pad, l, Z, o[128]
constexpr int kMaxCtas = 160;
constexpr float kNoMax = -1e38f;                  // reference of a part without tokens: finite, and below every other
constexpr float kSlack = 4.f;                     // logits may pass the reference by this much: weights up to 2^4

// Warps per CTA, one CTA per SM: what registers (128, 168 and 255 a thread, next to nothing spilled) and shared memory leave room
// for.  Fewer are slower: one query 16 warps 169 us, 12 warps 186 (4 bits 93.5 and 89.9); four queries 12 warps 67 us, 10 warps 78,
// 8 warps 72; eight queries 8 warps 104 us, 6 warps 136.
template <int NB>
__host__ __device__ constexpr int attend_warps() {
  return NB == 0 ? 16 : (NB == 1 ? 12 : 8);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_of_warp(float v) {  // one instruction; NaN is ignored
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Adds 1, ordered behind the warp's earlier writes and before its later reads (with a __syncwarp on either side).
__device__ __forceinline__ int add_acq_rel(int32_t* p) {
  int r;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(r) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const char* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zeros(uint32_t dst, const char* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed, for the whole warp
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
  __syncwarp();
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The codes of a word as pairs (j, j + P / 2) of fp16 subnormals: code 2^(kPairLow + pair_shift(j) - 24).  At 2 bits
// pairs 0 and 1 come from the word shifted up by 4 (by the multiplier, whose pipe is free), 2..4 from the word itself and
// 5..7 from the word shifted down by 6.
template <int BITS>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) {
  if constexpr (BITS == 2)
    return j < 2 ? (w * 16u) & (0x00300030u << (2 * j))
                 : (j < 5 ? w & (0x00300030u << (2 * (j - 2))) : (w >> 6) & (0x00300030u << (2 * (j - 5))));
  else
    return (j < 2 ? w : w >> 8) & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
}
template <int BITS>
constexpr int kPairLow = BITS == 2 ? 4 : 0;
// log2 of the factor code_pair leaves on pair j, past 2^kPairLow.
template <int BITS>
__device__ __forceinline__ constexpr int pair_shift(int j) {
  return BITS == 2 ? 2 * (j < 2 ? j : (j < 5 ? j - 2 : j - 5)) : 4 * (j & 1);
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
    s.len = a.lens[b];
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
  u.q_sink = min(nq, static_cast<int>((static_cast<uint32_t>(s.sink_end) + UT - 1) / UT));
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
    const int next = a.cu_tokens[b + 1];
    if (next == a.cu_tokens[b]) return -1;
    row = next - 1;
    if (a.positions != nullptr && row >= 0 && row < a.max_tokens && a.positions[row] < 0) return -1;
  }
  if (row < 0 || row >= a.q_rows) {
    *bad = true;
    return -1;
  }
  return row;
}

// Units per head of row i (0: it takes no query).
template <int UT>
__device__ __forceinline__ int row_units(const AttendArgs& a, int i) {
  bool bad = false;
  return q_row(a, i, &bad) < 0 ? 0 : units_of<UT>(span_of(a, i, &bad)).total;
}

// Where a warp is: unit `local` of a head (KV head and query pass he) of row seq.
struct Cursor {
  int seq, he, local;
  uint32_t f0;                  // of the split: the head's first unit (set for a head in hand)
  int row, q0, queries;  // row of q and out, first query head and queries of the pass
  Units un;
  Span sp;
};

// The cursor at unit `local` of a head, for the whole warp: {index, plain successors, block or its base, 1: residual + 2: ok}.
template <int UT>
__device__ __noinline__ int4 enter(const AttendArgs& a, Cursor& c, int seq, int he, int local, bool new_seq) {
  Units un;
  Span sp;
  int row;
  if (new_seq) {
    bool bad;
    sp = span_of(a, seq, &bad);
    un = units_of<UT>(sp);
    row = q_row(a, seq, &bad);
  } else {
    sp = c.sp;
    un = c.un;
    row = c.row;
  }
  const int h = a.passes == 1 ? he : he / a.passes, q0 = (he - h * a.passes) * a.per_pass;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    c.seq = seq;
    c.he = he;
    c.local = local;
    c.row = row;
    c.q0 = h * a.gqa + q0;
    c.queries = min(a.per_pass, a.gqa - q0);
    c.sp = sp;
    c.un = un;
  }
  __syncwarp();
  const bool res = local >= un.q_units;
  const int r = res ? local - un.q_units : local, sink = res ? un.r_sink : un.q_sink, gap = res ? un.r_gap : un.q_gap;
  const int end = res ? un.total - un.q_units : un.q_units, x = r + (r >= sink ? gap : 0);
  int4 out = make_int4(x, (r < sink ? sink : end) - r - 1, h, 2);
  if (res)  // not ok: the one unit of a row without tokens
    out.z = seq * a.heads + h, out.w = 1 + (x * kResTokens < sp.len - sp.quant ? 2 : 0);
  else if (a.block_table == nullptr)
    out.z = static_cast<int>((static_cast<uint32_t>(seq) * a.heads + h) * a.blocks_per_head);
  return out;
}
// The unit behind the last of a run of plain successors.
template <int UT>
__device__ __noinline__ int4 next_run(const AttendArgs& a, Cursor& c, int steps) {
  int seq = c.seq, he = c.he, local = c.local + steps;
  bool new_seq = false;
  if (local >= c.un.total) {
    local = 0;
    if (++he == a.heads * a.passes) {
      he = 0;
      new_seq = true;
      do ++seq;
      while (seq < a.rows - 1 && row_units<UT>(a, seq) == 0);
    }
  }
  return enter<UT>(a, c, seq, he, local, new_seq);
}

// A warp's shared memory.  NB: column blocks of four queries; 0: one query on byte digits.
template <int BITS, int NB>
struct __align__(128) WarpSmem {
  static constexpr int kQueries = NB == 0 ? 1 : 4 * NB;
  uint8_t k[kResTokens * kRow];
  uint8_t v[kResTokens * kRow];
  uint8_t q[2][kQueries * kQRow];     // raw queries: of the head in hand, and of the next one as it arrives
  uint4 p[NB == 0 ? 1 : NB][NB == 0 ? 32 : (BITS == 2 ? 128 : 64)];  // P operands
  uint4 qh[NB == 0 ? 1 : NB][NB == 0 ? 1 : 4][32];                   // Q operands (NB > 0: before s, each lane's share)
  uint4 zero4;                        // NB == 0: the operand of the other tile of a pair
  float part[kQueries * kPart];       // of the warp's first head, where that is not whole (of its last head: in k)
  Cursor cur, now, first;             // of the unit fetched last, of the head in hand, and of the warp's first head
  int partial;                        // bit 0: of its first head the warp has a part (in part), bit 1: of its last one (in k)
};
static_assert(kResTokens * kRow >= 4 * kVPieceStride && kResTokens * kRow >= kHalfBytes && kResTokens * kRow >= 8 * kPart * 4,
              "a buffer holds either kind of half, and the partials of a warp's last head");

// x / d with recip = floor((2^32 - 1) / d): the product's upper word is at most two short.
__device__ __forceinline__ uint32_t divide(uint32_t x, uint32_t d, uint32_t recip) {
  uint32_t q = __umulhi(x, recip), r = x - q * d;
  if (r >= d) r -= d, ++q;
  if (r >= d) ++q;
  return q;
}
// How `total` units are cut: worker w has those from start(w) on.  Workers of a CTA (`per_cta` of them) are neighbours.
struct Split {
  uint32_t total, workers, per_cta, len, longer;  // len units each, one more for the first `longer`
  uint32_t recip, recip1, recip_cta;              // of len, len + 1 and per_cta
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * len + min(w, longer); }
  __device__ __forceinline__ uint32_t worker_of(uint32_t f) const {
    const uint32_t cut = longer * (len + 1), more = f < cut ? 1 : 0;
    return (more ? 0 : longer) + divide(more ? f : f - cut, len + more, more ? recip1 : recip);
  }
};

// A warp's walk over its range of units: what is fetched when, where the halves land, and the ends of heads.  Core is the
// arithmetic: start_head, quant_k, quant_v, Res (state of residual rows) with res_start, res_k, res_v and res_end, finish.
template <int BITS, int NB, class Core>
struct Walker {
  static constexpr int P = 32 / BITS;                  // codes per word
  static constexpr int UT = attend_unit_tokens(BITS);  // tokens per quantized unit
  static constexpr int PT = UT / 4;                    // tokens of two V word rows
  using Smem = WarpSmem<BITS, NB>;
  static constexpr int NQ = Smem::kQueries;            // queries a warp holds

  const AttendArgs& a;
  Smem& S;
  const int lane, g, t;

  // the unit fetched last: its index among the row's units of codes or residual rows, how many plain successors it has,
  // whether it can be read, and where it is
  int x, run_, steps_;  // steps_: since the cursor was written
  bool res, ok, head;     // head: its K half brings the head's queries
  int slot;               // of S.q that the head fetched last has
  uint32_t blk, hbase;    // block; KV head (pages) or first block of the head (contiguous)
  long long off;          // bytes from the start of the K and V arrays
  const int32_t* table;   // the row's block table, or null
  int slot_now;           // of S.q that the head in hand has
  int full_from, sink_full;  // units from the one and below the other are visible whole

  __device__ Walker(const AttendArgs& args, Smem& smem, int ln) : a(args), S(smem), lane(ln), g(ln >> 2), t(ln & 3) {}

  // ---- units ---------------------------------------------------------------------------------------
  // Runs of plain successors are stepped through in registers; what changes at their ends is in shared memory.
  __device__ __forceinline__ void fetch_codes() {
    const uint32_t j = static_cast<uint32_t>(x) >> a.lg_upb;
    if (table != nullptr) {
      const int page = table[j];  // j < max_blocks: span_of
      ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages);
      blk = static_cast<uint32_t>(ok ? page : 0) * static_cast<uint32_t>(a.heads) + hbase;
    } else {
      ok = true;
      blk = hbase + j;
    }
    off = static_cast<long long>(static_cast<unsigned long long>(blk) * static_cast<uint32_t>(kHalfBytes << a.lg_upb) +
                                 (static_cast<uint32_t>(x) & ((1u << a.lg_upb) - 1)) * kHalfBytes);
  }
  __device__ __forceinline__ void fetch() {
    if (!res)
      fetch_codes();
    else
      off = static_cast<long long>(static_cast<unsigned long long>(blk) * static_cast<uint32_t>((kHeadDim * 2) << a.lg_r) +
                                   static_cast<uint32_t>(x) * kHalfBytes);
  }
  __device__ __forceinline__ void take(const int4& r) {
    x = r.x;
    run_ = r.y;
    res = r.w & 1;
    ok = (r.w & 2) != 0;
    head = S.cur.local == 0;
    if (res) {
      blk = static_cast<uint32_t>(r.z);
    } else {
      hbase = static_cast<uint32_t>(r.z);
      table = a.block_table == nullptr ? nullptr : a.block_table + static_cast<size_t>(S.cur.seq) * a.max_blocks;
    }
  }
  __device__ __forceinline__ void advance() {
    ++steps_;
    if (run_ > 0) {
      --run_;
      ++x;
      head = false;
    } else {
      take(next_run<UT>(a, S.cur, steps_));
      steps_ = 0;
    }
  }

  // Copies of a unit's halves, 16 bytes per lane and step; a group is committed whether or not there are any.
  __device__ __forceinline__ void copy_k_codes() {
    const uint32_t dst = smem_u32(S.k) + 16 * lane;
    const char* src = reinterpret_cast<const char*>(a.k_codes) + off + 16 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) copy16(dst + 512 * i, src + 512 * i);
  }
  __device__ __forceinline__ void copy_v_codes() {
    const uint32_t dst = smem_u32(S.v) + 16 * lane;
    const char* src = reinterpret_cast<const char*>(a.v_codes) + off + 16 * lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) copy16(dst + (i >> 1) * kVPieceStride + (i & 1) * 512, src + 512 * i);
  }
  __device__ __forceinline__ void bad_page() const {  // looked at when the copies are due, so that nothing waits for the page before
    if (lane == 0) report_status(a.status, KIVI_ERR_INTERNAL);
  }
  __device__ __forceinline__ void issue_k(bool any) {
    if (any && !ok && !res) bad_page();
    if (any && head) {  // NQ rows of 16 chunks (fewer queries: rows of zeros)
      slot ^= 1;
      const Cursor& c = S.cur;
      const char* src = reinterpret_cast<const char*>(a.q) + (static_cast<size_t>(c.row) * a.heads * a.gqa + c.q0) * (kHeadDim * 2);
#pragma unroll
      for (int i = 0; i < (NQ + 1) / 2; ++i) {
        const int qi = 2 * i + (lane >> 4);
        if (qi >= NQ) break;
        copy16_or_zeros(smem_u32(S.q[slot]) + qi * kQRow + (lane & 15) * 16, src + (qi < c.queries ? qi * 256 + (lane & 15) * 16 : 0),
                        qi < c.queries);
      }
    }
    if (any && ok) {
      if (!res) {
        copy_k_codes();
      } else {
        const uint32_t dst = smem_u32(S.k);
        const char* src = reinterpret_cast<const char*>(a.k_res) + off + 16 * lane;
#pragma unroll 1  // a loop, so that the paths stay branches and not sixteen predicated copies
        for (int i = 0; i < 8; ++i) copy16(dst + (lane >> 4) * kRow + (lane & 15) * 16 + 2 * kRow * i, src + 512 * i);
      }
    }
    copies_commit();
  }
  __device__ __forceinline__ void issue_v(bool any) {
    if (any && ok) {
      if (!res) {
        copy_v_codes();
      } else {
        const uint32_t dst = smem_u32(S.v);
        const char* src = reinterpret_cast<const char*>(a.v_res) + off + 16 * lane;
        const Span& n = S.cur.sp;
        const int tok = n.quant + x * kResTokens + (lane >> 4);
#pragma unroll 1  // hidden rows may hold anything: zeros instead
        for (int i = 0; i < 8; ++i)
          copy16_or_zeros(dst + (lane >> 4) * kRow + (lane & 15) * 16 + 2 * kRow * i, src + 512 * i, seen(n, tok + 2 * i));
      }
    }
    copies_commit();
  }
  // (s, z) of this lane's piece: K channels 32 t .. 32 t + 31 and V tokens PT t .. PT t + PT - 1
  __device__ __forceinline__ void load_pairs(uint32_t& kp, uint32_t& vp) const {
    if (ok && !res) load_code_pairs(kp, vp);
  }
  __device__ __forceinline__ void load_code_pairs(uint32_t& kp, uint32_t& vp) const {
    const uint32_t in = (static_cast<uint32_t>(x) & ((1u << a.lg_upb) - 1)) * UT;
    const size_t ks = static_cast<unsigned long long>(blk) * static_cast<uint32_t>(kHeadDim >> a.lg_gk) + ((32 * t) >> a.lg_gk);
    const size_t vs = static_cast<unsigned long long>(blk) * (1u << (a.lg_r - a.lg_gv)) + ((in + PT * t) >> a.lg_gv);
    kp = static_cast<uint32_t>(a.k_scale[ks]) | (static_cast<uint32_t>(a.k_zero[ks]) << 16);
    vp = static_cast<uint32_t>(a.v_scale[vs]) | (static_cast<uint32_t>(a.v_zero[vs]) << 16);
  }
  __device__ static __forceinline__ bool seen(const Span& n, int tok) {
    return tok < n.len && (tok < n.sink_end || tok >= n.start);
  }

  // ---- heads that several warps share ----------------------------------------------------------------------------
  // Partials (m, l, Z and o[128] of each query) are joined by log-sum-exp: those of a CTA's warps in shared memory when all of
  // them are done, a warp per head and query, and those of several CTAs in global memory by the warp that arrives last at the
  // ticket of the head and query.  Parts are taken in their order, so the result does not depend on who arrives when.
  struct Sums {
    float m, l, Z, o[4];  // channels 4 lane .. 4 lane + 3
  };
  __device__ static __forceinline__ void store_row(uint16_t* out, int lane, const Sums& s) {
    const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
    *reinterpret_cast<uint2*>(out + 4 * lane) =
        make_uint2(pack_h2((s.o[0] + s.Z) * inv, (s.o[1] + s.Z) * inv), pack_h2((s.o[2] + s.Z) * inv, (s.o[3] + s.Z) * inv));
  }
  // s joined with the n <= 32 parts at p0, p + stride, p + 2 stride, ..: lane i weighs part i, so that the rows follow without
  // a chain of maxima.  GLOBAL: past the L1 cache, which may hold what was there before.
  template <bool GLOBAL>
  __device__ static __forceinline__ float4 part_of(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p);
    return GLOBAL ? __ldcg(q) : *q;
  }
  template <bool GLOBAL>
  __device__ static __forceinline__ void add_parts(Sums& s, int lane, const float* p0, const float* p, int stride, int n) {
    float4 x = make_float4(kNoMax, 0.f, 0.f, 0.f);
    if (lane < n) x = part_of<GLOBAL>(lane == 0 ? p0 : p + lane * stride);
    const float mn = fmaxf(s.m, max_of_warp(x.x)), f = ex2(s.m - mn), w = ex2(x.x - mn);
    s.m = mn;
    s.l *= f;
    s.Z *= f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s.o[e] *= f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 v = part_of<GLOBAL>((i == 0 ? p0 : p + i * stride) + 4 + 4 * lane);
      const float wi = __shfl_sync(kFull, w, i);
      s.l = fmaf(wi, __shfl_sync(kFull, x.z, i), s.l);
      s.Z = fmaf(wi, __shfl_sync(kFull, x.w, i), s.Z);
      s.o[0] = fmaf(wi, v.x, s.o[0]);
      s.o[1] = fmaf(wi, v.y, s.o[1]);
      s.o[2] = fmaf(wi, v.z, s.o[2]);
      s.o[3] = fmaf(wi, v.w, s.o[3]);
    }
  }
  // By every warp of the CTA, behind a barrier.  The loops are kept small: this code comes from a cold instruction cache.
  __device__ __noinline__ static void join(const AttendArgs& a, const Smem* warps, const Split& sp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, count = static_cast<int>(blockDim.x >> 5);
    const uint32_t lo = blockIdx.x * sp.per_cta, cta_start = sp.start(min(lo, sp.workers));
    const uint32_t cta_end = sp.start(min(lo + sp.per_cta, sp.workers));
    // candidate 2 w + k: warp w's first (k = 0) or last head, where it has only a part of it and is the first of the CTA to
    static_assert(2 * attend_warps<NB>() <= 32, "a lane looks at one of them");
    bool lead = false;
    if (lane < 2 * count) {
      const Smem& S = warps[lane >> 1];
      const Cursor& c = lane & 1 ? S.now : S.first;
      lead = (S.partial >> (lane & 1) & 1) != 0 && (lane < 2 || c.f0 >= sp.start(lo + (lane >> 1)));
    }
    const unsigned leads = __ballot_sync(kFull, lead);
    const int heads = __popc(leads);
#pragma unroll 1
    for (int task = warp; task < heads * a.per_pass; task += count) {
      const int k = task / a.per_pass, q = task - k * a.per_pass;
      unsigned rest = leads;
      for (int i = 0; i < k; ++i) rest &= rest - 1;
      const int at = __ffs(rest) - 1, w0 = at >> 1;
      const Cursor& c = at & 1 ? warps[w0].now : warps[w0].first;
      if (q >= c.queries) continue;
      const uint32_t f0 = c.f0, f1 = f0 + c.un.total;
      // its parts: this one, and the first heads of the warps behind it
      const bool mine = lane >= w0 && lane < static_cast<int>(sp.per_cta) && lo + lane < sp.workers && sp.start(lo + lane) < f1;
      const int n = __popc(__ballot_sync(kFull, mine));
      const float* part0 = (at & 1 ? reinterpret_cast<const float*>(warps[w0].k) : warps[w0].part) + q * kPart;
      Sums s = {kNoMax, 0.f, 0.f, {0.f, 0.f, 0.f, 0.f}};
      add_parts<false>(s, lane, part0, warps[w0].part + q * kPart, sizeof(Smem) / sizeof(float), n);
      uint16_t* out = a.out + (static_cast<size_t>(c.row) * a.heads * a.gqa + c.q0 + q) * kHeadDim;
      if (f0 >= cta_start && f1 <= cta_end) {
        store_row(out, lane, s);
        continue;
      }
      // a CTA's partial heads: the one it starts in (slot 0) and the one it ends in
      float* to = a.partials + (static_cast<size_t>(2 * blockIdx.x + (cta_start >= f0 ? 0 : 1)) * NQ + q) * kPart;
      if (lane == 0) *reinterpret_cast<float4*>(to) = make_float4(s.m, 0.f, s.l, s.Z);
      *reinterpret_cast<float4*>(to + 4 + 4 * lane) = make_float4(s.o[0], s.o[1], s.o[2], s.o[3]);
      __syncwarp();  // every lane's share of the partial comes before the ticket
      const uint32_t b0 = f0 >= cta_start ? blockIdx.x : divide(sp.worker_of(f0), sp.per_cta, sp.recip_cta);
      const uint32_t b1 = f1 <= cta_end ? blockIdx.x : divide(sp.worker_of(f1 - 1), sp.per_cta, sp.recip_cta);
      const size_t ticket = (static_cast<size_t>(c.seq) * a.heads * a.passes + c.he) * a.per_pass + q;
      int last = 0;
      if (lane == 0) last = add_acq_rel(a.tickets + ticket) == static_cast<int>(b1 - b0);
      if (!__shfl_sync(kFull, last, 0)) continue;
      __syncwarp();
      if (lane == 0) a.tickets[ticket] = 0;
      const int parts = static_cast<int>(b1 - b0) + 1, stride = 2 * NQ * kPart;
      const float* part_i = a.partials + (2 * static_cast<size_t>(b0) * NQ + q) * kPart;
      const float* part_0 = part_i + (sp.start(b0 * sp.per_cta) >= f0 ? 0 : NQ * kPart);
      s = {kNoMax, 0.f, 0.f, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 1
      for (int i0 = 0; i0 < parts; i0 += 32)
        add_parts<true>(s, lane, i0 == 0 ? part_0 : part_i + i0 * stride, part_i + i0 * stride, stride, min(32, parts - i0));
      store_row(out, lane, s);
    }
  }

  // worker: of the split; seq0: row of its first unit, the row's units before it: rem.
  __device__ __forceinline__ void run(const Split& split, uint32_t worker, int seq0, uint32_t rem) {
    Core& core = static_cast<Core&>(*this);
    const uint32_t f0 = split.start(worker);
    int left = static_cast<int>(split.start(worker + 1) - f0);
    {
      bool bad;
      const uint32_t n = units_of<UT>(span_of(a, seq0, &bad)).total, he = rem / n;
      take(enter<UT>(a, S.cur, seq0, static_cast<int>(he), static_cast<int>(rem - he * n), true));
      steps_ = 0;
      slot = 0;
      head = true;
    }
    fetch();
    issue_k(true);
    issue_v(true);
    uint32_t kp = 0, vp = 0;
    load_pairs(kp, vp);
    uint32_t at = f0;
    while (left > 0) {
      const Cursor& c = S.cur;
      const int l0 = c.local, units = c.un.total;
      const int count = min(left, units - l0), nq = min(count, max(0, c.un.q_units - l0));
      __syncwarp();
      if (lane == 0) {
        S.now = c;
        S.now.f0 = at - l0;
        if (at == f0) S.first = S.now;
      }
      __syncwarp();
      slot_now = slot;
      full_from = static_cast<int>((static_cast<uint32_t>(S.now.sp.start) + UT - 1) / UT);
      sink_full = S.now.sp.sink_end / UT;
      copies_wait<1>();  // the head's queries are here with its first K half
      core.start_head();
      // K of the unit in hand, then V; the next unit's K is copied behind the one, its V behind the other
#pragma unroll 1
      for (int i = 0; i < nq; ++i) {
        const int ux = x;
        const bool good = ok, more = --left > 0;
        const uint32_t ckp = kp, cvp = vp;
        const bool plain = i + 1 < nq && run_ > 0;  // the next unit is the next one of the same codes: nothing else to look at
        if (plain) {
          --run_;
          ++steps_;
          ++x;
          fetch_codes();
        } else if (more) {
          advance();
          fetch();
        }
        copies_wait<1>();
        if (good) core.quant_k(ux, ckp, cvp);
        __syncwarp();  // the K half has been read, and the P operands are written
        if (plain) {
          if (ok) {
            copy_k_codes();
            load_code_pairs(kp, vp);
          } else {
            bad_page();
          }
          copies_commit();
        } else {
          issue_k(more);
          if (more) load_pairs(kp, vp);
        }
        copies_wait<1>();
        if (good) core.quant_v();
        __syncwarp();
        if (plain) {
          if (ok) copy_v_codes();
          copies_commit();
        } else {
          issue_v(more);
        }
      }
      if (count > nq) {
        typename Core::Res r;
        core.res_start(r);
#pragma unroll 1
        for (int i = nq; i < count; ++i) {
          const int ux = x;
          const bool good = ok, more = --left > 0;
          if (more) {
            advance();
            fetch();
          }
          copies_wait<1>();
          if (good) core.res_k(ux, r);
          __syncwarp();
          issue_k(more);
          if (more) load_pairs(kp, vp);
          copies_wait<1>();
          if (good) core.res_v(r);
          __syncwarp();
          issue_v(more);
        }
        core.res_end(r);
      }
      const bool whole = count == units;
      if (whole) {
        core.finish(nullptr);
      } else if (at == f0) {
        core.finish(S.part);
        if (lane == 0) S.partial |= 1;
      } else {  // the last head: no copy is in flight any more
        core.finish(reinterpret_cast<float*>(S.k));
        if (lane == 0) S.partial |= 2;
      }
      at += count;
    }
  }
};

// Several queries per KV head: fp16 products, two columns per query (top of the file).
template <int BITS, int NB>
struct Many : Walker<BITS, NB, Many<BITS, NB>> {
  using Base = Walker<BITS, NB, Many<BITS, NB>>;
  using Base::a, Base::S, Base::lane, Base::g, Base::t, Base::slot_now, Base::full_from, Base::sink_full;
  using Base::UT, Base::PT, Base::P, Base::NQ, Base::seen;
  static constexpr int HP = P / 2;                  // code pairs per word
  static constexpr int MT = UT / 16;                // K tiles per unit
  static constexpr int KW = kHeadDim / P / 4;       // K words per lane and token
  // V codes are at bit 4 or above of their halves (code 2^-20): the lost bits of lower ones (top of the file) show most where
  // sum_t p_t z takes most of the sum back.  At 2 bits code_pair has them there; at 4 bits quant_v puts all at bits 4..7.  K codes at
  // 4 bits stay at bits 0..7: lifting them costs 4% (88 -> 92 us) for an error of 1.4e-5 instead of 1.7e-5, beside a rounding of 2.1e-4.
  static constexpr int kVUp = 4;
  struct Res {
    float p[NB][2], r[NB][8][4];
  };

  // state of the head in hand: lane (g, t) is query t (of each column block) and channels 16 g .. 16 g + 15.
  // Weights are 2^(logit - m): m is the largest logit when it was last raised, by at most kSlack below the largest.
  float m[NB], thr[NB], l[NB], Z[NB], o[NB][8][4];
  float qs[NB][4];   // scale * log2 e * sum of q over channels 32 i .. 32 i + 31
  int qe[NB];        // exponent of the largest |q|
  float vf[NB];      // of the unit in hand: what its sums of P operands and V codes are times, to join o

  using Base::Base;

  // ---- the head's queries ----------------------------------------------------------------------------
  __device__ void start_head() {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint4 v[4];
      const uint4* src = reinterpret_cast<const uint4*>(S.q[slot_now] + (4 * b + (g >> 1)) * kQRow + 64 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = src[i];
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
      uint32_t qh[16];
#pragma unroll
      for (int x = 0; x < KW; ++x)
#pragma unroll
        for (int j = 0; j < HP; ++j) {
          const float sc = pow2i(6 - e - pair_shift<BITS>(j));
          qh[x * HP + j] = pack_h2(f[x * P + j] * sc, f[x * P + j + HP] * sc);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) S.qh[b][i][lane] = make_uint4(qh[4 * i], qh[4 * i + 1], qh[4 * i + 2], qh[4 * i + 3]);
      qe[b] = __shfl_sync(kFull, e, 8 * t);
#pragma unroll
      for (int i = 0; i < 4; ++i) qs[b][i] = a.qscale * __shfl_sync(kFull, sum, 8 * t + i);
      m[b] = 0.f;
      thr[b] = -INFINITY;  // any logit sets the reference
      l[b] = Z[b] = 0.f;
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[b][v8][i] = 0.f;
    }
    __syncwarp();
  }

  // The largest of a query's lanes.
  __device__ __forceinline__ static float max_of_query(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
    return fmaxf(x, __shfl_xor_sync(kFull, x, 16));
  }
  // Where a logit (over m) passes the threshold, m moves up to the largest (the first time: to wherever that is), and
  // o, l and Z with it.  Returns how far m moved.
  __device__ __forceinline__ float raise(int b, float mu) {
    const float mx = max_of_query(mu);
    if (!(mx > thr[b])) return 0.f;
    thr[b] = kSlack;
    m[b] += mx;
    const float al = ex2(-fmaxf(mx, 0.f));  // the first time o, l and Z are zero
    l[b] *= al;
    Z[b] *= al;
#pragma unroll
    for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[b][v8][i] *= al;
    return mx;
  }

  // Slot of P operand vector (column n, code pair jl of word rows of lane tt): conflict-free for the
  // lanes that write one (jl and tt fixed by g, columns 2 t + lo) and those that read it (n = g, tt = t).
  __device__ static __forceinline__ int p_slot(int n, int jl, int tt) {
    return n * 16 + ((jl * 4 + tt) ^ ((n >> 1) | ((n & 1) << 2)));
  }

  // ---- K half of a quantized unit: logits, softmax, P operands ------------------------------------------
  // Tile i = (tb, x, jj) (2 bits) or (tb, x) holds on rows g and g + 8 the tokens of pair j = 4 jj + g % 4 (g % 4)
  // of word row 2 tt + x, tt = 2 (g / 4) + tb: what lane tt of the V product needs as one operand register.
  __device__ __forceinline__ void quant_k(int ux, uint32_t kp, uint32_t vp) {
    const int jl = g & 3, tt0 = (g >> 2) * 2, tok0 = ux * UT;
    const bool full = ux >= full_from || ux < sink_full;
    if (!full) {  // V pieces that are hidden whole have no say (their s and z may be anything)
      const int p0 = tok0 + PT * t;
      if (p0 >= S.now.sp.sink_end && p0 + PT <= S.now.sp.start) vp = 0;
    }
    const unsigned ksm = __reduce_max_sync(kFull, kp & 0xFFFFu);
    const int ek = max(1, static_cast<int>(ksm >> 10));
    const __half2 sh = __float2half2_rn(h2f(static_cast<uint16_t>(kp)) * pow2i(22 - ek));
    const __half2 nsh = (g & 1) ? __hneg2(sh) : __float2half2_rn(0.f);
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = h2f(static_cast<uint16_t>(__shfl_sync(kFull, kp, i) >> 16));
    uint32_t kb[NB][16];
    float inv[NB], cst[NB], lg[NB][MT][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 q4 = S.qh[b][i][lane];
        const uint32_t w[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kb[b][4 * i + j] = as_u32(__hfma2(as_h2(w[j]), sh, __hmul2(as_h2(w[j]), nsh)));  // even columns: q s rounded; odd: the rest
      }
      inv[b] = a.qscale * pow2i(qe[b] + ek - 4 - kPairLow<BITS>);
      cst[b] = fmaf(z[3], qs[b][3], fmaf(z[2], qs[b][2], fmaf(z[1], qs[b][1], z[0] * qs[b][0]))) - m[b];
    }
    const uint8_t* kt = S.k + ((g >> 2) * (UT / 2) + jl) * (16 * BITS) + 4 * KW * t;
    // two tiles at a time: two independent chains of sums per column block
#pragma unroll
    for (int i0 = 0; i0 < MT; i0 += 2) {
      uint32_t w[2][2][KW];  // [tile][row g, g + 8][word]
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = i0 + i;
        const int off = BITS == 2 ? (n >> 2) * 1024 + ((n >> 1) & 1) * 512 + (n & 1) * 128 : (n >> 1) * 1024 + (n & 1) * 512;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if constexpr (BITS == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(kt + off + 256 * y);
            w[i][y][0] = x.x, w[i][y][1] = x.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(kt + off + 256 * y);
            w[i][y][0] = x.x, w[i][y][1] = x.y, w[i][y][2] = x.z, w[i][y][3] = x.w;
          }
        }
      }
      float c[2][NB][4];
#pragma unroll
      for (int x = 0; x < KW; ++x) {
#pragma unroll
        for (int j = 0; j < HP; j += 2)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a0 = code_pair<BITS>(w[i][0][x], j), a1 = code_pair<BITS>(w[i][1][x], j);
            const uint32_t a2 = code_pair<BITS>(w[i][0][x], j + 1), a3 = code_pair<BITS>(w[i][1][x], j + 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              if (x == 0 && j == 0)
                mma16_first(c[i][b], a0, a1, a2, a3, kb[b][0], kb[b][1]);
              else
                mma16(c[i][b], a0, a1, a2, a3, kb[b][x * HP + j], kb[b][x * HP + j + 1]);
            }
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          lg[b][i0 + i][0] = fmaf(c[i][b][0] + c[i][b][1], inv[b], cst[b]);
          lg[b][i0 + i][1] = fmaf(c[i][b][2] + c[i][b][3], inv[b], cst[b]);
        }
    }
    if (!full) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int tok = BITS == 2 ? tok0 + 32 * (tt0 + (i >> 2)) + 16 * ((i >> 1) & 1) + 4 * (i & 1) + jl
                                  : tok0 + 16 * (tt0 + (i >> 1)) + 8 * (i & 1) + jl;
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (!seen(S.now.sp, tok + HP * y))
#pragma unroll
            for (int b = 0; b < NB; ++b) lg[b][i][y] = -INFINITY;
      }
    }
    constexpr int HALF = MT / 2;  // tiles of one tb
    float mu[NB][2];
    bool above = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        mu[b][tb] = fmaxf(lg[b][tb * HALF][0], lg[b][tb * HALF][1]);
#pragma unroll
        for (int i = 1; i < HALF; ++i) mu[b][tb] = fmaxf(mu[b][tb], fmaxf(lg[b][tb * HALF + i][0], lg[b][tb * HALF + i][1]));
      }
      above = above || fmaxf(mu[b][0], mu[b][1]) > thr[b];
    }
    if (__any_sync(kFull, above)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float by = raise(b, fmaxf(mu[b][0], mu[b][1]));
        mu[b][0] -= by;
        mu[b][1] -= by;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          lg[b][i][0] -= by;
          lg[b][i][1] -= by;
        }
      }
    }
    const uint32_t vq[2] = {__shfl_sync(kFull, vp, tt0), __shfl_sync(kFull, vp, tt0 + 1)};
    const float vs[2] = {h2f(static_cast<uint16_t>(vq[0])), h2f(static_cast<uint16_t>(vq[1]))};
    constexpr int JJ = BITS == 2 ? 2 : 1;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // operands from 2^14 to 2^15 for the largest p s; 2^-80 and less (weights are up to 2^kSlack) count as nothing
      const float top = max_of_query(fmaxf(ex2(mu[b][0]) * vs[0], ex2(mu[b][1]) * vs[1]));
      const int e = min(max(__float_as_int(top) >> 23, 127 - 80), 127 + 121);
      const float up = pow2i(14 + 127 - e);
      vf[b] = pow2i(e - 127 - 14 + 24 - kVUp);
      float fac[2][JJ];
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        const float s = vs[tb] * up;
        if constexpr (BITS == 2) {
          fac[tb][0] = s * pow2i(-pair_shift<2>(jl));
          fac[tb][1] = s * pow2i(-pair_shift<2>(jl + 4));
        } else {
          fac[tb][0] = s;
        }
      }
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        uint32_t hi[HALF], lo[HALF];
        float ps = 0.f;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
          const float p0 = ex2(lg[b][tb * HALF + i][0]), p1 = ex2(lg[b][tb * HALF + i][1]);
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
  // A k chunk takes the two pairs that one 8-byte part of a P vector holds: pairs jl and jl + 4 of word row x (2 bits),
  // pair jl of both word rows (4 bits).
  __device__ __forceinline__ void quant_v() {
    uint32_t pb[NB][4][BITS == 2 ? 4 : 2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int jl = 0; jl < 4; ++jl) {
        if constexpr (BITS == 2) {
          const uint4 x = S.p[b][p_slot(g, jl, t)];
          pb[b][jl][0] = x.x, pb[b][jl][1] = x.y, pb[b][jl][2] = x.z, pb[b][jl][3] = x.w;
        } else {
          const uint2 x = reinterpret_cast<const uint2*>(S.p[b])[p_slot(g, jl, t)];
          pb[b][jl][0] = x.x, pb[b][jl][1] = x.y;
        }
      }
    // The sums of a unit start from zero and join o by rounded additions: the tensor cores cut sums off, and over a long
    // sequence of positive terms, most of which sum_t p_t z then takes back, that would show.
    const uint8_t* vt = S.v + t * kVPieceStride + 64 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint4 w4 = *reinterpret_cast<const uint4*>(vt + x * 512 + 16 * i);
        w[x][0] = w4.x, w[x][1] = w4.y, w[x][2] = w4.z, w[x][3] = w4.w;
      }
      float c[2][NB][4];
      auto product = [&](bool first, int e, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, int jl, int x) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (first)
            mma16_first(c[e / 2][b], a0, a1, a2, a3, pb[b][jl][2 * x], pb[b][jl][2 * x + 1]);
          else
            mma16(c[e / 2][b], a0, a1, a2, a3, pb[b][jl][2 * x], pb[b][jl][2 * x + 1]);
        }
      };
#pragma unroll
      for (int jl = 0; jl < 4; ++jl) {
        if constexpr (BITS == 2) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint32_t v0 = w[x][e], v1 = w[x][e + 1];
              product(jl == 0 && x == 0, e, code_pair<2>(v0, jl), code_pair<2>(v1, jl), code_pair<2>(v0, jl + 4), code_pair<2>(v1, jl + 4),
                      jl, x);
            }
        } else {
          auto pair = [&](uint32_t v) { return (jl == 0 ? v * 16u : (jl == 1 ? v : v >> (jl == 2 ? 4 : 8))) & 0x00F000F0u; };
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            product(jl == 0, e, pair(w[0][e]), pair(w[0][e + 1]), pair(w[1][e]), pair(w[1][e + 1]), jl, 0);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q) o[b][2 * i + e][q] = fmaf(c[e][b][q], vf[b], o[b][2 * i + e][q]);
    }
  }

  // ---- residual units, on the tensor cores too: K rows with the raw queries, V rows transposed on the way ----------
  // Logits of rows g and g + 8 for query t, as weights times 2^10 in p.
  __device__ __forceinline__ void res_start(Res& s) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8) s.r[b][v8][0] = s.r[b][v8][1] = s.r[b][v8][2] = s.r[b][v8][3] = 0.f;
  }
  __device__ __forceinline__ void res_k(int ux, Res& s) {
    float(&p)[NB][2] = s.p;
    float(&r)[NB][8][4] = s.r;
    float c[NB][4];
    const uint32_t row = smem_u32(S.k) + (lane & 15) * kRow + (lane >> 4) * 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t x[4];
      ldmatrix4(x, row + 32 * i);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(S.q[slot_now] + (4 * b + (g >> 1)) * kQRow) + 8 * i + t;
        const uint32_t b0 = (g & 1) ? 0u : q[0], b1 = (g & 1) ? 0u : q[4];
        if (i == 0)
          mma16_first(c[b], x[0], x[1], x[2], x[3], b0, b1);
        else
          mma16(c[b], x[0], x[1], x[2], x[3], b0, b1);
      }
    }
    const int tok0 = S.now.sp.quant + ux * kResTokens;
    const bool s0 = seen(S.now.sp, tok0 + g), s1 = seen(S.now.sp, tok0 + g + 8);
    bool above = false;
    float mu[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      p[b][0] = s0 ? fmaf(c[b][0], a.qscale, -m[b]) : -INFINITY;
      p[b][1] = s1 ? fmaf(c[b][2], a.qscale, -m[b]) : -INFINITY;
      mu[b] = fmaxf(p[b][0], p[b][1]);
      above = above || mu[b] > thr[b];
    }
    if (__any_sync(kFull, above)) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float by = raise(b, mu[b]), al = ex2(-fmaxf(by, 0.f));
        p[b][0] -= by;
        p[b][1] -= by;
#pragma unroll
        for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
          for (int i = 0; i < 4; ++i) r[b][v8][i] *= al;
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      p[b][0] = ex2(p[b][0]);
      p[b][1] = ex2(p[b][1]);
      l[b] += p[b][0] + p[b][1];
      p[b][0] *= 1024.f;
      p[b][1] *= 1024.f;
    }
  }
  // r: tile v8 holds channels 16 v8 + g (row g) and 16 v8 + 8 + g (row g + 8), columns as o; times 2^10.
  __device__ __forceinline__ void res_v(Res& s) {
    const float(&p)[NB][2] = s.p;
    float(&r)[NB][8][4] = s.r;
    uint32_t pb[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __shfl_sync(kFull, p[b][i >> 1], 4 * (2 * t + (i & 1)) + (g >> 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t hi = pack_h2(x[2 * i], x[2 * i + 1]);
        const float2 f = unpack_h2(hi);
        pb[b][i] = (g & 1) ? pack_h2(x[2 * i] - f.x, x[2 * i + 1] - f.y) : hi;
      }
    }
    const uint32_t row = smem_u32(S.v) + ((lane & 7) + (lane >> 4) * 8) * kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int v8 = 0; v8 < 8; ++v8) {
      uint32_t x[4];
      ldmatrix4_trans(x, row + 32 * v8);
#pragma unroll
      for (int b = 0; b < NB; ++b) mma16(r[b][v8], x[0], x[1], x[2], x[3], pb[b][0], pb[b][1]);
    }
  }
  // The residual rows' share of the output, through shared memory to the layout of o.
  __device__ __forceinline__ void res_end(Res& s) {
    const float(&r)[NB][8][4] = s.r;
    float* buf = reinterpret_cast<float*>(S.p[0]);  // 4 queries at a time of 64 channels: 1 KB
    constexpr float f = 1.f / 1024.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          buf[64 * t + 16 * v + g] = (r[b][4 * half + v][0] + r[b][4 * half + v][1]) * f;
          buf[64 * t + 16 * v + 8 + g] = (r[b][4 * half + v][2] + r[b][4 * half + v][3]) * f;
        }
        __syncwarp();
        if ((g >> 2) == half) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(buf + 64 * t + 16 * (g & 3) + 4 * i);
            o[b][2 * i][0] += x.x;
            o[b][2 * i][2] += x.y;
            o[b][2 * i + 1][0] += x.z;
            o[b][2 * i + 1][2] += x.w;
          }
        }
      }
    __syncwarp();
  }

  // ---- the end of a head's segment -----------------------------------------------------------------------
  // Lane (g, t): o of query t (each column block), channels 16 g .. 16 g + 15.
  __device__ __forceinline__ void finish(float* part) {
    const int nq = S.now.queries;
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
        f[2 * v8] = o[b][v8][0] + o[b][v8][1];
        f[2 * v8 + 1] = o[b][v8][2] + o[b][v8][3];
      }
      if (part == nullptr) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack_h2((f[2 * i] + zs) * inv, (f[2 * i + 1] + zs) * inv);
        uint4* dst = reinterpret_cast<uint4*>(
            a.out + (static_cast<size_t>(S.now.row) * a.heads * a.gqa + S.now.q0 + qi) * kHeadDim + 16 * g);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        float* dst = part + qi * kPart;
        if (g == 0) *reinterpret_cast<float4*>(dst) = make_float4(ls == 0.f ? kNoMax : m[b], 0.f, ls, zs);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(dst + 4 + 16 * g + 4 * i) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
      }
    }
  }
};

// ---- one query per KV head: exact integer products of code bytes and byte digits -----------------------------------------
// With one query the columns of the fp16 scheme stay mostly empty, and its masks (nine per 2-bit word) set the time.  Here the
// A operand of mma m16n8k32 (u8 x s8, int32 sums) takes a code word as it is and its copies without the lowest codes of each
// byte: V_k = sum over i >= k of c_i 2^(b i), k = 0 .. P / 4 - 1, one AND per copy but the first.  Against
// X_k = W (Q_k 2^(-b k) - Q_(k-1) 2^(-b (k-1))), W = 2^(b (P / 4 - 1)), the products add up to W sum c_k Q_k, exactly.  Q is
// q_c s_g(c), P is p_t s_g(t), as fixed point relative to the largest of the block (23 bits) or of the unit (24 bits); each X
// (below 2^30) is four signed byte digits, one B column each.  Two tiles of 16 tokens (or channels) share a sum: the digits of
// the one sit in columns 0..3, of the other in columns 4..7, each against zeros for the other tile.
constexpr float kQFixed = 8388544.f;   // 2^23 - 64
constexpr float kPFixed = 16777088.f;  // 2^24 - 128

__device__ __forceinline__ void mma_bytes(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bytes_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int BITS>
struct One : Walker<BITS, 0, One<BITS>> {
  using Base = Walker<BITS, 0, One<BITS>>;
  using Base::a, Base::S, Base::lane, Base::g, Base::t, Base::slot_now, Base::full_from, Base::sink_full;
  using Base::UT, Base::PT, Base::P, Base::seen;
  static constexpr int NV = P / 4;            // copies of a word: 4 at 2 bits, 2 at 4 bits
  static constexpr int W = 1 << (BITS * (NV - 1));
  static constexpr int TJ = UT / 32;          // tokens per lane and unit
  struct Res {
    float p[2], r[8][4];
  };

  // Lane holds the queries of the channels whose digits it forms: P word + NV m + k, word = lane / NV, k = lane % NV, m = 0..3
  // (K piece lane / 8), and channels 4 lane .. 4 lane + 3 of the output; l and Z are this lane's share.
  float q[4], qsum, m, l, Z, o[4];
  float alpha, invv;

  using Base::Base;

  __device__ __forceinline__ void start_head() {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(S.q[slot_now]) + P * (lane / NV) + (lane % NV);
    qsum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[i] = h2f(src[NV * i]) * a.qscale;
      qsum += q[i];
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) qsum += __shfl_xor_sync(kFull, qsum, off);  // of the piece's 32 channels
    m = kNoMax;
    l = Z = o[0] = o[1] = o[2] = o[3] = 0.f;
    if (lane == 0) S.zero4 = make_uint4(0, 0, 0, 0);
    __syncwarp();
  }

  // Digits of four values: digit d of x[i] in byte i of word d, from the bytes of x + 0x80808080, each less 128.
  __device__ static __forceinline__ void digits(const int (&x)[4], uint32_t (&wd)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = static_cast<uint32_t>(x[i]) + 0x80808080u;
    const uint32_t t0 = __byte_perm(u[0], u[1], 0x5140), t1 = __byte_perm(u[0], u[1], 0x7362);
    const uint32_t t2 = __byte_perm(u[2], u[3], 0x5140), t3 = __byte_perm(u[2], u[3], 0x7362);
    wd[0] = __byte_perm(t0, t2, 0x5410) ^ 0x80808080u;
    wd[1] = __byte_perm(t0, t2, 0x7632) ^ 0x80808080u;
    wd[2] = __byte_perm(t1, t3, 0x5410) ^ 0x80808080u;
    wd[3] = __byte_perm(t1, t3, 0x7632) ^ 0x80808080u;
  }
  // Operand words of code word i (a K word, or a V word row), copy k and column c (digit 3 - c): a lane t of the products
  // reads those of words NK t .. NK t + NK - 1 as 16-byte vectors; the XOR puts its four lanes t in four bank groups.
  __device__ static __forceinline__ uint32_t* operand(uint4* rows, int row, int c) {
    return reinterpret_cast<uint32_t*>(rows) + 16 * row + 4 * (c ^ ((row >> 1) & 3));
  }
  // Two digit columns of a tile end in each lane; the partner lane has the other two.  Even lanes t keep row g, odd lanes
  // row g + 8, whole (every digit sum is below 2^22).
  __device__ __forceinline__ float gather(const int (&c)[4]) const {
    const bool odd = t & 1;
    const float sc = odd ? 1.f : 65536.f;
    const float fg = static_cast<float>(c[0] * 256 + c[1]) * sc, fh = static_cast<float>(c[2] * 256 + c[3]) * sc;
    return (odd ? fh : fg) + __shfl_xor_sync(kFull, odd ? fg : fh, 1);
  }
  // Copies of the words of rows g and g + 8 against the operands of one word: W sum c Q of both rows, onto c or (first) alone.
  template <bool FIRST>
  __device__ static __forceinline__ void products(int (&c)[4], uint32_t wg, uint32_t wh, const uint4& b, int half) {
    const uint32_t b0 = BITS == 2 || half == 0 ? b.x : b.z, b1 = BITS == 2 || half == 0 ? b.y : b.w;
    const uint32_t mask = BITS == 2 ? 0xFCFCFCFCu : 0xF0F0F0F0u;
    if constexpr (FIRST)
      mma_bytes_first(c, wg, wh, wg & mask, wh & mask, b0, b1);
    else
      mma_bytes(c, wg, wh, wg & mask, wh & mask, b0, b1);
    if constexpr (BITS == 2) mma_bytes(c, wg & 0xF0F0F0F0u, wh & 0xF0F0F0F0u, wg & 0xC0C0C0C0u, wh & 0xC0C0C0C0u, b.z, b.w);
  }

  __device__ __forceinline__ void quant_k(int ux, uint32_t kp, uint32_t vp) {
    const bool full = ux >= full_from || ux < sink_full;
    const int tok0 = ux * UT;
    if (!full) {  // V pieces that are hidden whole have no say (their s and z may be anything)
      const int p0 = tok0 + PT * t;
      if (p0 >= S.now.sp.sink_end && p0 + PT <= S.now.sp.start) vp = 0;
    }
    // Q operands of the block
    const uint32_t kq = __shfl_sync(kFull, kp, lane >> 3);
    const float s = h2f(static_cast<uint16_t>(kq));
    float big = 0.f, cst = h2f(static_cast<uint16_t>(kq >> 16)) * qsum, v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = q[i] * s;
      big = fmaxf(big, fabsf(v[i]));
    }
    big = max_of_warp(big);
    cst += __shfl_xor_sync(kFull, cst, 8);
    cst += __shfl_xor_sync(kFull, cst, 16);
    const float fix = big > 0.f ? kQFixed * reciprocal(big) : 0.f, inv = big * (1.0f / (W * kQFixed));
    {
      const int k = lane % NV, xa = W >> (BITS * k), xb = k ? (W << BITS) >> (BITS * k) : 0;
      int xs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int Q = __float2int_rn(v[i] * fix), below = __shfl_up_sync(kFull, Q, 1);
        xs[i] = Q * xa - below * xb;
      }
      uint32_t wd[4];
      digits(xs, wd);
#pragma unroll
      for (int c = 0; c < 4; ++c) operand(S.qh[0][0], lane >> 2, c)[lane & 3] = wd[3 - c];
    }
    __syncwarp();
    // logits: pair j, tile b holds on row g + 8 c token P r + NV j' .. of word row r = g / 4 + 2 c + 4 b, so that after the
    // exchange lane (g, t) has tokens of word row g / 4 + 2 (t % 2) + 4 (t / 2): those whose P digits it forms
    float lg[TJ];
    {
      const int si = 8 * t + ((g & 3) ^ t);
      const uint4 *pe = g < 4 ? &S.qh[0][0][si] : &S.zero4, *po = g >= 4 ? &S.qh[0][0][si] : &S.zero4;
      const uint4 be[2] = {pe[0], pe[g < 4 ? 4 : 0]}, bo[2] = {po[0], po[g >= 4 ? 4 : 0]};
      const uint8_t* kt = BITS == 2 ? S.k + (16 * (g >> 2) + (g & 3)) * 32 + 8 * t
                                    : S.k + (8 * (g >> 2) + 4 * ((g >> 1) & 1) + (g & 1)) * 64 + 16 * t;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        int c[4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint8_t* r0 = kt + 128 * j + 2048 * b;
          const uint4& B0 = b ? bo[0] : be[0];
          const uint4& B1 = b ? bo[1] : be[1];
          if constexpr (BITS == 2) {
            const uint2 wg = *reinterpret_cast<const uint2*>(r0), wh = *reinterpret_cast<const uint2*>(r0 + 1024);
            if (b == 0)
              products<true>(c, wg.x, wh.x, B0, 0);
            else
              products<false>(c, wg.x, wh.x, B0, 0);
            products<false>(c, wg.y, wh.y, B1, 0);
          } else {
            const uint4 wg = *reinterpret_cast<const uint4*>(r0), wh = *reinterpret_cast<const uint4*>(r0 + 1024);
            if (b == 0)
              products<true>(c, wg.x, wh.x, B0, 0);
            else
              products<false>(c, wg.x, wh.x, B0, 0);
            products<false>(c, wg.y, wh.y, B0, 1);
            products<false>(c, wg.z, wh.z, B1, 0);
            products<false>(c, wg.w, wh.w, B1, 1);
          }
        }
        lg[j] = fmaf(gather(c), inv, cst);
      }
    }
    const int r = (g >> 2) + 2 * (t & 1) + 4 * (t >> 1);
    const int k = BITS == 2 ? g & 3 : g & 1, in = BITS == 2 ? k : 4 * ((g >> 1) & 1) + k;  // first token within the row
    if (!full) {
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        if (!seen(S.now.sp, tok0 + P * r + in + NV * j)) lg[j] = -INFINITY;
    }
    // softmax, and P operands relative to the unit's largest p s (2^-100 and less count as nothing)
    float mu = lg[0];
#pragma unroll
    for (int j = 1; j < TJ; ++j) mu = fmaxf(mu, lg[j]);
    const uint32_t vq = __shfl_sync(kFull, vp, r >> 1);
    const float vs = h2f(static_cast<uint16_t>(vq)), mn = fmaxf(m, max_of_warp(mu));
    alpha = ex2(m - mn);
    m = mn;
    const float top = max_of_warp(ex2(mu - mn) * vs);
    const bool some = top > 0x1p-100f;
    const float f = some ? kPFixed * reciprocal(top) * vs : 0.f;
    invv = some ? top * (1.0f / (W * kPFixed)) : 0.f;
    const int xa = W >> (BITS * k), xb = k ? (W << BITS) >> (BITS * k) : 0;
    float ps = 0.f;
    int xs[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const float p = ex2(lg[j] - mn);
      ps += p;
      const int Pf = static_cast<int>(__float2uint_rn(p * f)), below = __shfl_up_sync(kFull, Pf, 4);
      xs[j] = Pf * xa - below * xb;
    }
    l = fmaf(l, alpha, ps);
    Z = fmaf(Z, alpha, ps * h2f(static_cast<uint16_t>(vq >> 16)));
    uint32_t wd[4];
    digits(xs, wd);
    if constexpr (BITS == 2) {
#pragma unroll
      for (int c = 0; c < 4; ++c) operand(S.p[0], r, c)[k] = wd[3 - c];
    } else {  // bytes 2 mu and 2 mu + 1 of the words of row r, copy k: row pairs are the vectors
      const int mu2 = (g >> 1) & 1;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        reinterpret_cast<uint16_t*>(reinterpret_cast<uint32_t*>(S.p[0]) + 16 * (r >> 1) + 4 * (c ^ (r >> 1)) + 2 * (r & 1) + k)[mu2] =
            static_cast<uint16_t>(wd[3 - c]);
    }
  }

  // Pair v: tile b holds on row g + 8 c channel 16 g + 8 b + 4 c + v; lane (g, t) reads V word rows 2 t and 2 t + 1.
  __device__ __forceinline__ void quant_v() {
    uint4 be[2], bo[2];
    if constexpr (BITS == 2) {
      const int si = 8 * t + ((g & 3) ^ t);
      const uint4 *pe = g < 4 ? &S.p[0][si] : &S.zero4, *po = g >= 4 ? &S.p[0][si] : &S.zero4;
      be[0] = pe[0], be[1] = pe[g < 4 ? 4 : 0], bo[0] = po[0], bo[1] = po[g >= 4 ? 4 : 0];
    } else {
      const uint4 x = S.p[0][4 * t + ((g & 3) ^ t)], none = make_uint4(0, 0, 0, 0);
      be[0] = be[1] = g < 4 ? x : none;
      bo[0] = bo[1] = g >= 4 ? x : none;
    }
    int c[4][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint8_t* row = S.v + t * kVPieceStride + x * 512 + 64 * g;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint4 lo = *reinterpret_cast<const uint4*>(row + 32 * b), hi = *reinterpret_cast<const uint4*>(row + 32 * b + 16);
        const uint4& B = b ? bo[x] : be[x];
        const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          if (x == 0 && b == 0)
            products<true>(c[v], wl[v], wh[v], B, x);
          else
            products<false>(c[v], wl[v], wh[v], B, x);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) o[v] = fmaf(o[v], alpha, gather(c[v]) * invv);
  }

  // ---- residual rows: fp16 products as for several queries, every column the one query --------------------------------
  __device__ __forceinline__ void res_start(Res& s) const {
#pragma unroll
    for (int v8 = 0; v8 < 8; ++v8) s.r[v8][0] = s.r[v8][1] = s.r[v8][2] = s.r[v8][3] = 0.f;
  }
  __device__ __forceinline__ void res_k(int ux, Res& s) {
    float c[4];
    const uint32_t row = smem_u32(S.k) + (lane & 15) * kRow + (lane >> 4) * 16;
    const uint32_t* qw = reinterpret_cast<const uint32_t*>(S.q[slot_now]) + t;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t x[4];
      ldmatrix4(x, row + 32 * i);
      if (i == 0)
        mma16_first(c, x[0], x[1], x[2], x[3], qw[0], qw[4]);
      else
        mma16(c, x[0], x[1], x[2], x[3], qw[8 * i], qw[8 * i + 4]);
    }
    const int tok0 = S.now.sp.quant + ux * kResTokens;
    const float l0 = seen(S.now.sp, tok0 + g) ? c[0] * a.qscale : -INFINITY;
    const float l1 = seen(S.now.sp, tok0 + g + 8) ? c[2] * a.qscale : -INFINITY;
    const float mn = fmaxf(m, max_of_warp(fmaxf(l0, l1)));
    if (mn > m) {  // the same for every lane
      const float al = ex2(m - mn);
      m = mn;
      l *= al;
      Z *= al;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= al;
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8)
#pragma unroll
        for (int i = 0; i < 4; ++i) s.r[v8][i] *= al;
    }
    const float p0 = ex2(l0 - mn), p1 = ex2(l1 - mn);
    if (t == 0) l += p0 + p1;  // lanes t hold the same rows
    s.p[0] = p0 * 1024.f;
    s.p[1] = p1 * 1024.f;
  }
  __device__ __forceinline__ void res_v(Res& s) {
    uint32_t pb[2];
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __shfl_sync(kFull, s.p[i >> 1], 4 * (2 * t + (i & 1)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t hi = pack_h2(x[2 * i], x[2 * i + 1]);
      const float2 f = unpack_h2(hi);
      pb[i] = (g & 1) ? pack_h2(x[2 * i] - f.x, x[2 * i + 1] - f.y) : hi;
    }
    const uint32_t row = smem_u32(S.v) + ((lane & 7) + (lane >> 4) * 8) * kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
    for (int v8 = 0; v8 < 8; ++v8) {
      uint32_t w[4];
      ldmatrix4_trans(w, row + 32 * v8);
      mma16(s.r[v8], w[0], w[1], w[2], w[3], pb[0], pb[1]);
    }
  }
  __device__ __forceinline__ void res_end(Res& s) {
    float* buf = reinterpret_cast<float*>(S.p[0]);  // 128 channels
    __syncwarp();
    if (t == 0) {
#pragma unroll
      for (int v8 = 0; v8 < 8; ++v8) {
        buf[16 * v8 + g] = (s.r[v8][0] + s.r[v8][1]) * (1.f / 1024.f);
        buf[16 * v8 + 8 + g] = (s.r[v8][2] + s.r[v8][3]) * (1.f / 1024.f);
      }
    }
    __syncwarp();
    const float4 x = *reinterpret_cast<const float4*>(buf + 4 * lane);
    o[0] += x.x;
    o[1] += x.y;
    o[2] += x.z;
    o[3] += x.w;
    __syncwarp();
  }

  __device__ __forceinline__ void finish(float* part) {
    const typename Base::Sums s = {m, warp_sum(l), warp_sum(Z), {o[0], o[1], o[2], o[3]}};
    if (part == nullptr) {
      Base::store_row(a.out + (static_cast<size_t>(S.now.row) * a.heads * a.gqa + S.now.q0) * kHeadDim, lane, s);
    } else {
      if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(s.l == 0.f ? kNoMax : m, 0.f, s.l, s.Z);
      *reinterpret_cast<float4*>(part + 4 + 4 * lane) = make_float4(o[0], o[1], o[2], o[3]);
    }
  }
};

template <int BITS, int NB>
struct CoreOf {
  using type = Many<BITS, NB>;
};
template <int BITS>
struct CoreOf<BITS, 0> {
  using type = One<BITS>;
};

template <int BITS, int NB>
__global__ void __launch_bounds__(attend_warps<NB>() * 32, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  after_previous_kernel();
  constexpr int W = attend_warps<NB>(), T = W * 32, UT = CoreOf<BITS, NB>::type::UT;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Smem = WarpSmem<BITS, NB>;
  __shared__ int warp_sum[W], cum[T + 1];  // units per head before each thread's rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.rows + T - 1) / T, r0 = min(a.rows, tid * per), r1 = min(a.rows, r0 + per);
  int mine = 0;
  for (int i = r0; i < r1; ++i) {
    bool bad = false;
    if (q_row(a, i, &bad) >= 0) (void)span_of(a, i, &bad);
    if (bad && blockIdx.x == 0) report_status(a.status, KIVI_ERR_INTERNAL);
    mine += row_units<UT>(a, i);
  }
  int x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(kFull, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  const int active = __syncthreads_count(mine > 0) * per;  // rows with a query, at most
  int before = x - mine;
  for (int i = 0; i < warp; ++i) before += warp_sum[i];
  cum[tid] = before;
  if (tid == T - 1) cum[T] = before + mine;
  __syncthreads();
  const uint32_t he_count = static_cast<uint32_t>(a.heads) * a.passes;
  Split split;
  split.total = static_cast<uint32_t>(cum[T]) * he_count;  // below 2^32: checked on the host
  if (split.total == 0) return;
  // Few units are spread over the SMs, but no further than pays: parts of a head that lie in one CTA join in shared memory, those of
  // several through tickets and global memory, which the last to arrive reads one after another.  A head of no more units than warps
  // stays in a CTA, a longer one is cut into halves of a CTA unless that makes more than 20 parts.  One sequence, 2 bits, calls in a row,
  // against a unit per CTA: 1024 tokens x 4 heads 12.7 -> 11.0 us, 2048 x 1 12.9 -> 12.2, 8192 x 1 19.9 -> 12.6 (R = 512 21.4 -> 12.7,
  // four queries 19.8 -> 12.8), 32000 x 1 26.5 -> 15.1, 4 bits 16000 x 1 25.5 -> 14.3; what loses is 4 sequences of up to 1000 x 8:
  // 12.0 -> 12.5, and 16 of up to 300 x 2: 11.3 -> 11.5.  Without the limit of 20: 32000 x 1 16.1, but 8192 x 1 12.1.
  split.per_cta = min(static_cast<uint32_t>(W), (split.total + gridDim.x - 1) / gridDim.x);
  if (split.per_cta < W) {
    const uint32_t per_head = (static_cast<uint32_t>(cum[T]) + active - 1) / static_cast<uint32_t>(active);
    uint32_t parts = per_head <= W ? 1 : (per_head + W / 2 - 1) / (W / 2);
    if (parts > 20) parts = (per_head + W - 1) / W;
    split.per_cta = max(split.per_cta, (per_head + parts - 1) / parts);  // at most W
  }
  split.workers = min(split.total, gridDim.x * split.per_cta);
  split.len = split.total / split.workers;
  split.longer = split.total - split.len * split.workers;
  split.recip = 0xffffffffu / split.len;
  split.recip1 = 0xffffffffu / (split.len + 1);
  split.recip_cta = 0xffffffffu / split.per_cta;
  const uint32_t worker = blockIdx.x * split.per_cta + warp;
  Smem* warps = reinterpret_cast<Smem*>(smem_raw);
  if (lane == 0) warps[warp].partial = 0;
  if (warp < split.per_cta && worker < split.workers) {
    // the row of the worker's first unit: its thread's rows by bisection, then one by one
    const uint32_t f0 = split.start(worker);
    const int want = static_cast<int>(f0 / he_count);
    int lo = 0, hi = T;  // cum[lo] <= want < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= want)
        lo = mid;
      else
        hi = mid;
    }
    int row = lo * per, first = cum[lo];
    for (int n; first + (n = row_units<UT>(a, row)) <= want; ++row) first += n;
    typename CoreOf<BITS, NB>::type d(a, warps[warp], lane);
    d.run(split, worker, row, f0 - first * he_count);
  }
  __syncthreads();
  CoreOf<BITS, NB>::type::join(a, warps, split);
}

template <int BITS, int NB>
cudaError_t launch(const AttendArgs& a, int ctas, cudaStream_t stream) {
  constexpr int smem = attend_warps<NB>() * static_cast<int>(sizeof(WarpSmem<BITS, NB>));
  static_assert(smem + 4 * (attend_warps<NB>() * 33 + 1) <= 232448 - 1024, "a CTA holds 227 KB of shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(attend_kernel<BITS, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(attend_kernel<BITS, NB>, dim3(ctas), attend_warps<NB>() * 32, smem, stream, a);
}

struct Shape {
  int passes, per_pass, blocks;  // query passes per KV head, queries of a pass, column blocks of four (0: one query)
};
Shape shape_of(int gqa) {
  Shape s;
  s.passes = (gqa + 7) / 8;
  s.per_pass = (gqa + s.passes - 1) / s.passes;
  s.blocks = s.per_pass > 4 ? 2 : (gqa > 1 ? 1 : 0);
  return s;
}
// A workspace is the partials of any call, then the tickets: calls of other caches and numbers of query heads may use it one after
// the other, since none of them writes partials where another one looks for its tickets, which each leaves zero.
constexpr size_t kPartialBytes = static_cast<size_t>(kMaxCtas) * 2 * 8 * kPart * sizeof(float);
static_assert(kPartialBytes % 256 == 0, "tickets behind the partials");
size_t ticket_bytes(long long rows, int heads, const Shape& s) {
  return (static_cast<size_t>(rows) * heads * s.passes * s.per_pass * sizeof(int32_t) + 255) & ~static_cast<size_t>(255);
}

}  // namespace

size_t attend_workspace_bytes(long long rows, int heads, int gqa, long long max_units) {
  const Shape s = shape_of(gqa);
  if (rows * max_units > 0xffffffffll / (static_cast<long long>(heads) * s.passes)) return 0;
  return kPartialBytes + ticket_bytes(rows, heads, s);
}

cudaError_t launch_attend(AttendArgs a, int bits, void* workspace, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const Shape s = shape_of(a.gqa);
  a.passes = s.passes;
  a.per_pass = s.per_pass;
  a.lg_upb = a.lg_r - (bits == 2 ? 7 : 6);
  a.partials = static_cast<float*>(workspace);
  a.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + kPartialBytes);
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int n = sms < kMaxCtas ? sms : kMaxCtas;
  if (bits == 2) return s.blocks == 0 ? launch<2, 0>(a, n, stream) : (s.blocks == 1 ? launch<2, 1>(a, n, stream) : launch<2, 2>(a, n, stream));
  return s.blocks == 0 ? launch<4, 0>(a, n, stream) : (s.blocks == 1 ? launch<4, 1>(a, n, stream) : launch<4, 2>(a, n, stream));
}

}  // namespace kivi
