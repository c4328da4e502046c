// Attention over the paged 8-bit cache on the tensor cores (tcgen05), for
// bf16 queries and heads of up to 128 dimensions.
//
// The cached codes go from HBM to the MMAs as they are: no kernel instruction
// touches a key or a value.  What has to meet them in 8 bits is the small
// side, split so that nothing is lost:
//   q    is scaled by a power of two and written as the sum of two 8-bit
//        numbers (8 bits, all that bf16 has), both products added: E4M3 and,
//        of what that leaves, E4M3 again of 2^5 times it where the two scores
//        stand side by side, E5M2 where they fall onto the same columns.  (In
//        E4M3 as it is, which ends at 2^-9, small values would lose all below
//        2^-10.)  So a value is exact to 2^-21 of the largest of the rows that
//        share a scale.  The rows of a unit do; a row more than 2^4 below the
//        largest has its own, so that every row has 2^-17 of its own largest
//        (one more multiplication a score: 36 rows 73.5 -> 77.7 us, 72 rows
//        97.1 -> 107.0 us, 96 rows 111.5 -> 124.2 us, eight sequences of
//        16,384, which is why not all rows do);
//   P    the softmax weights are written as the sum of four E5M2 numbers, in
//        all exact to 2^-13 of themselves or 2^-16, whichever is more: E5M2
//        has nothing below 2^-16, which is 2^-25 of the row's largest weight in
//        this run at worst (that one lies above 2^9).  The sum of the weights
//        counts them as they are in fp32, so n weights of less than 2^-26 of
//        the largest, which the products drop, pull the output towards 0 by n
//        2^-26 of the values' size at most.  E5M2 is the upper byte of fp16:
//        of the weight rounded to fp16 a part is that byte after rounding, the
//        rest an exact fp16 difference, and three parts of three bits and a
//        sign hold its eleven bits; the fourth is the upper byte of what fp16
//        rounded off.  That takes no conversion to 8 bits (parts made by those
//        took 1200 cycles a tile of 80 rows), and no part needs a scale of its
//        own.  Without the fourth part: 2^-11, and 2 to 7 % less time.
// Scores are computed transposed: S^T[token, row] = K q^T and
// O^T[dim, row] = V^T P^T, so that the 128 lanes of an MMA are always full
// (tokens, then dimensions) and the number of (query, head) rows, a multiple
// of 16 up to 96, is the MMA's N: the cost follows the rows there are.  A
// thread of the softmax owns one token: its key's and its value's scale are
// one factor and one addend in the exponent (the value's scale, a power of
// two, rides on the weight).  So a score's exponent is rounded at the size of
// the two together: to 2^-18 with values of 2^64, where fp32 has 2^-21 for a
// score of 8 alone.  Adding the scale to the reference first would spare that
// and cost 1 to 2.6 % of the time with 72 rows.
//   V^T is the V tile as it lies (dimensions contiguous), an A operand with M
//   contiguous; P^T is written by token, 16 rows to a 16-byte unit, a B
//   operand with N contiguous.
// The running maximum is lazy: weights are taken against a reference that is
// raised (and the accumulators rescaled, by an exact power of two) only when
// a token beats it by more than 2^5.75; fp16 has room for that.
//
// Work is split by tiles of 128 tokens: all tiles of all (sequence, key head,
// row tile) units are numbered, and each CTA (one per SM) takes an equal run
// of them, whatever the sequences' lengths; a unit that is cut leaves partial
// sums that a second launch joins.
//
// Warps: 0 copies tiles (TMA, one box per page), 1 issues the MMAs, 2-3 lay
// out q, the others do the softmax (groups of four, one per lane quarter; a
// group has 8 or 16 rows) and write the output.  Every wait is bounded; on a timeout the CTA
// stops issuing, drains, frees TMEM and flags the error word.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kernels.h"
#include "tc_ptx.cuh"

namespace dflash {
namespace {

constexpr int kTile = 128;         // tokens of a tile, lanes of an MMA
constexpr int kMaxRows = 96;       // (query, head) rows of a unit
constexpr int kMaxCtas = 160;
constexpr int kUnitBytes = kTile * 128;  // a K or V tile in shared memory
constexpr int kStages = 7;         // most stages of K or V tiles
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHead = 10.f;      // weights are 2^(score - ref + kHead)
// A row's sum counts its weights without their value scales (2^lv), times
// 2^kSumRef: with scales from 2^kLeastLv to 2^kMostLv and 2^30 tokens it stays
// between 2^-95 and 2^126, whichever of them the reference has come from.
constexpr float kSumRef = 16.f;
constexpr float kLeastLv = -64.f, kMostLv = 120.f;
// Weights of pages whose value scale is that much (in bits) below the largest
// of the run so far may underflow: their terms of the sum are computed apart.
constexpr float kFarLv = 90.f;
constexpr float kRaise = 15.75f;   // 2^15.75 = 55109 < 57344, E5M2's largest
constexpr int kUnitCost = 4;       // of a unit besides its tiles, in tiles
constexpr int kParts = 4;          // E5M2 parts of a weight
constexpr int kRowsApart = 4;      // bits below the unit's: a scale of its own

// Shared-memory plan for N rows.
template <int N>
struct Plan {
  static constexpr int Q = 2 * N * 128;           // two parts of q
  static constexpr int P = 2 * kParts * N * 128;  // two buffers
  // softmax groups: as many as registers allow (a group's warp on each SM
  // quarter hides the others' latencies), in whole rows of 16, eights or
  // fours
  static constexpr int kGroups = N >= 64 ? 4 : N == 48 ? 3 : 2;
  static constexpr int kRowsOf = N / kGroups;           // rows of a group
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kFixed = 7 * 1024 + 1024;  // Meta, alignment
  static constexpr int kFit = (232448 - Q - P - kFixed) / kUnitBytes;
  // K is free again after the first product, V after the second
  static constexpr int K = kFit / 2 - 1 < 5 ? kFit / 2 - 1 : 5;
  static constexpr int V = kFit - K < kStages ? kFit - K : kStages;
  static constexpr int kBytes = kFixed + Q + P + (K + V) * kUnitBytes;
  // The parts of an operand lie side by side in the MMA's N where it (256)
  // and TMEM (512 columns) allow: fewer MMAs, whose time is that of reading
  // the 128 lanes' operand when N is small.
  static constexpr int kScore = N <= 64 ? 2 * N : N;    // columns of a tile
  static constexpr int kAcc = N <= 64 ? kParts * N : 2 * N;
  // Of q's second part: its factor (undone where the scores are added) and type
  static constexpr float kRestUp = kScore == 2 * N ? 32.f : 1.f;
  static constexpr __nv_fp8_interpretation_t kRestType =
      kScore == 2 * N ? __NV_E4M3 : __NV_E5M2;
  static constexpr int kUse = 2 * kScore + kAcc;
  static constexpr int kCols =
      kUse <= 128 ? 128 : kUse <= 256 ? 256 : 512;
};

// One unit's part that a CTA works on, with what its rows need.
struct Segment {
  int done;                // no more work
  int b, hk, row0;         // first row of the row tile
  int t0, t1;              // tiles
  int n, nq;               // cached tokens, queries
  int whole, slot;         // all of the unit's tiles / where partial sums go
  int min_lim;             // tokens that every live row sees
  alignas(16) int lim[kMaxRows];     // tokens each row sees
  alignas(16) float rel[kMaxRows];   // undoes a row's own scaling
  float back;                        // undoes the unit's
  int uneven;                        // some row has its own scaling
  int out_row[kMaxRows];             // row of out and lse, -1: none
  int on[kMaxRows];                  // the row has a query
};

struct Meta {
  Segment seg[2];
  alignas(16) float neg_ref[kMaxRows], fac[kMaxRows];
  float q_top[2];
  alignas(16) float warp_val[4][kMaxRows];
  // of a page: key factor, log2 of the value scale, 2^(kSumRef - that) or 0
  float ct[kStages][8], lv[kStages][8], fl[kStages][8];
  uint64_t kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages];
  uint64_t sfull[2], pfull[2], qfull[2], qempty[2], qfree;
  uint64_t drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Meta) <= 7 * 1024, "");

// ---- the numbering of the tiles -------------------------------------------
struct Shape {
  int N, row_tiles, rows, g;  // rows = Q * g
};
struct Lens {
  int n, nq;
};
__device__ __forceinline__ Lens lens_of(const PagedAttnArgs& a, int b,
                                        bool* bad) {
  Lens l;
  l.n = attn_clamp(a.kv_len[b], (long long)a.max_pages * a.page, bad);
  l.nq = attn_clamp(a.q_len ? a.q_len[b] : a.Q, a.Q, bad);
  return l;
}
// Tiles that row tile rt of a sequence needs (0: it sees nothing).
__device__ __forceinline__ int tiles_of(const PagedAttnArgs& a, const Shape& s,
                                        const Lens& l, int rt) {
  if (s.row_tiles == 1) return l.nq > 0 ? (l.n + kTile - 1) / kTile : 0;
  const int q0 = rt * s.N / s.g;
  if (q0 >= l.nq) return 0;
  int seen = l.n;
  if (a.causal) {
    const int q1 = min((min((rt + 1) * s.N, s.rows) - 1) / s.g, l.nq - 1);
    seen = max(0, min(l.n, l.n - l.nq + q1 + 1));
  }
  return (seen + kTile - 1) / kTile;
}
// Work of one key head of a sequence, in tiles: every unit counts kUnitCost
// more than its tiles (its start and its output take about that long), so
// that a run of short sequences does not fall to one CTA.
// Fewer than 2^31 in all (checked on the host).
__device__ __forceinline__ int head_work(const PagedAttnArgs& a,
                                         const Shape& s, const Lens& l) {
  int w = 0;
  for (int rt = 0; rt < s.row_tiles; ++rt) w += kUnitCost + tiles_of(a, s, l, rt);
  return w;
}
// First position of CTA c of the G that work.
__device__ __forceinline__ int run_start(int total, int c, int G) {
  const int q = total / G;
  return c >= G ? total : q * c + (total - q * G) * c / G;
}

// Walks the units from a position in the numbering.  Position kUnitCost + t
// of a unit is its tile t; a unit without tiles is at its last position.
struct Walk {
  int b, hk, rt, at;         // at: position in the unit
  int left;                  // positions left in this CTA's run
  int first;                 // no segment handed out yet
  int total, G;              // all positions, and the CTAs that work
};
// A unit that is cut, for the join: CTA c leaves it here if the unit's first
// tile is CTA c - 1's and its next is c's own.
struct alignas(16) Cut {
  int b, hk, rt;
  int parts;  // 0: no such unit; 2 n + odd: n parts, the first in the odd slot
};
// Words of partial sums, before the CTAs' Cuts.
__host__ __device__ constexpr size_t part_words(int grid, int N) {
  return (size_t)2 * grid * N * (128 + 2);
}
// Where the run of CTA `cta` of `grid` starts.  A whole warp, each lane with
// a stretch of the sequences; *bad: some length was out of range.
__device__ void walk_start(const PagedAttnArgs& a, const Shape& s, int cta,
                           int grid, Walk& w, bool* bad) {
  const int lane = threadIdx.x & 31;
  const int per = (a.B + 31) / 32;
  const int b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
  int work = 0;
  for (int b = b0; b < b1; ++b)
    work += a.Hkv * head_work(a, s, lens_of(a, b, bad));
  int run = work;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  const int total = __shfl_sync(0xffffffffu, run, 31);
  const int G = min(grid, total);
  const int p0 = run_start(total, cta, G), p1 = run_start(total, cta + 1, G);
  w.left = p1 - p0;
  w.first = 1;
  w.total = total;
  w.G = G;
  w.b = w.hk = w.rt = w.at = 0;
  if (w.left <= 0) return;                 // the same in every lane
  const bool mine = p0 >= run - work && p0 < run;
  int o = p0 - (run - work), h = 1;
  if (mine) {
    for (w.b = b0; w.b < b1; ++w.b) {
      h = head_work(a, s, lens_of(a, w.b, bad));
      if (o < a.Hkv * h) break;
      o -= a.Hkv * h;
    }
    w.hk = o / h;
    o -= w.hk * h;
    const Lens l = lens_of(a, w.b, bad);
    for (;; ++w.rt) {
      const int t = kUnitCost + tiles_of(a, s, l, w.rt);
      if (o < t) break;
      o -= t;
    }
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  w.b = __shfl_sync(0xffffffffu, w.b, from);
  w.hk = __shfl_sync(0xffffffffu, w.hk, from);
  w.rt = __shfl_sync(0xffffffffu, w.rt, from);
  w.at = __shfl_sync(0xffffffffu, o, from);
}
// What CTA `cta` leaves for the join, from the start of its walk.
__device__ __forceinline__ Cut cut_at(const PagedAttnArgs& a, const Shape& s,
                                      const Walk& w, int cta) {
  Cut c{w.b, w.hk, w.rt, 0};
  if (w.left <= 0 || w.at <= kUnitCost) return c;  // no tile lies before
  bool bad = false;
  const int before = run_start(w.total, cta, w.G) - w.at;  // first position
  const int head = before + kUnitCost;                     // its first tile's
  const int end = head + tiles_of(a, s, lens_of(a, w.b, &bad), w.rt);
  const int c0 = (int)(((head + 1ll) * w.G - 1) / w.total);
  if (c0 != cta - 1) return c;
  const int c1 = (int)(((long long)end * w.G - 1) / w.total);
  // a run's first segment is in its even slot; every part but the first
  // starts its run, and the first does if no unit before it ends there
  c.parts = 2 * (c1 - c0 + 1) + (run_start(w.total, c0, w.G) < before);
  return c;
}
struct Part {
  int b, hk, rt, t0, t1, whole, first;
  Lens l;
};
// The next segment; false at the end of the run.
__device__ bool walk_next(const PagedAttnArgs& a, const Shape& s, Walk& w,
                          Part& p) {
  bool bad = false;
  while (w.left > 0) {
    p.l = lens_of(a, w.b, &bad);
    const int t = tiles_of(a, s, p.l, w.rt);
    const int work = kUnitCost + t;
    const int end = min(work, w.at + w.left);
    p.b = w.b;
    p.hk = w.hk;
    p.rt = w.rt;
    p.t0 = max(0, w.at - kUnitCost);
    p.t1 = max(0, end - kUnitCost);
    p.whole = p.t0 == 0 && p.t1 == t;
    w.left -= end - w.at;
    w.at = end;
    if (end == work) {
      w.at = 0;
      if (++w.rt == s.row_tiles) {
        w.rt = 0;
        if (++w.hk == a.Hkv) {
          w.hk = 0;
          ++w.b;
        }
      }
    }
    if (p.t1 > p.t0 || (t == 0 && end == work)) {
      p.first = w.first;
      w.first = 0;
      return true;
    }
  }
  return false;
}

// Wait for phase `parity` of `bar`, at most `limit` ns; false (and *abort set)
// if it runs out or another role gave up.  Polls go to shared memory, whose
// bandwidth the MMAs need: the clock and *abort are looked at every 64 polls
// (some 100 us; every poll with a limit below a millisecond), and roles that
// run ahead (kLazy) sleep between polls.
template <bool kLazy = false>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity,
                                         volatile int* abort,
                                         uint64_t limit) {
  if (tc::mbar_try_wait(bar, parity, 1000)) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  const int polls = limit < 1000000ull ? 1 : 64;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < polls; ++i) {
      if (kLazy) __nanosleep(100);
      if (tc::mbar_try_wait(bar, parity, 1000)) return true;
    }
    if (*abort) return false;
    if (tc::globaltimer_ns() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
}

// Position in a ring of S stages; `phase` flips on every lap.
template <int S>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == S) {
      at = 0;
      phase ^= 1;
    }
  }
  // the stage k (<= S) uses back
  __device__ __forceinline__ Ring back(int k) const {
    Ring r = *this;
    r.at -= k;
    if (r.at < 0) {
      r.at += S;
      r.phase ^= 1;
    }
    return r;
  }
};

// ---- PTX ------------------------------------------------------------------
// Instruction descriptor of the second product: E4M3 x E5M2 (format 1 in
// bits 10-12) -> fp32, both operands with M / N contiguous (bits 15, 16).
__host__ __device__ constexpr uint32_t idesc_mn(int N) {
  return tc::idesc_e4m3_f32(128, N) | (1u << 10) | (1u << 15) | (1u << 16);
}
// M contiguous in 128-byte rows with 128-byte swizzle (a V tile as TMA
// writes it): groups of eight tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return tc::sdesc_k_sw128(saddr);  // the same fields: stride 1024, swizzle
}
// N contiguous in 16-byte units, no swizzle: groups of eight tokens 128
// bytes apart (leading offset), groups of 16 rows 2048 apart (stride).
__device__ __forceinline__ uint64_t sdesc_mn_plain(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(2048 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}
__device__ __forceinline__ void tmem_ld4(uint32_t addr, float* v) {
  uint32_t r[4];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
          addr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
      "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
      : "memory");
}
// Wait for this thread's TMEM loads; no use of v is scheduled before it.
template <int M>
__device__ __forceinline__ void tmem_loaded(float (&v)[M]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < M; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                   tc::smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src,
                                       bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(read ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Barrier `id` of T threads; true if `p` is true in any of them.
template <int T>
__device__ __forceinline__ bool any_of(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "n"(T)
      : "memory");
  return r != 0;
}
constexpr int kQBar = 15;  // of the two warps that lay out q
__device__ __forceinline__ bool half_any(int id, bool p) {
  return any_of<128>(id, p);
}
__device__ __forceinline__ void half_sync(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(id) : "memory");
}

// Largest of the warp's values.
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Sums over the warp's lanes of C values each, by halves: the lanes trade
// half of what they hold as long as that is even.  Value i ends in v[0..] of
// the lanes `slot`, the first value that this lane holds, says.
template <int C, int O>
__device__ __forceinline__ void lane_sums(float* v, int lane, int& slot) {
  if constexpr (O > 0) {
    if constexpr (C % 2 == 0) {
      const bool up = lane & O;
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const float give = up ? v[i] : v[i + C / 2];
        const float keep = up ? v[i + C / 2] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
      }
      if (up) slot += C / 2;
      lane_sums<C / 2, O / 2>(v, lane, slot);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        v[i] += __shfl_xor_sync(0xffffffffu, v[i], O);
      lane_sums<C, O / 2>(v, lane, slot);
    }
  }
}
// Values a lane holds in the end.
constexpr int lane_share(int C, int O) {
  return O == 0 ? C : lane_share(C % 2 ? C : C / 2, O / 2);
}
// One thread of the warp (always the same one).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r != 0;
}

// Pairs of fp32 in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Four weights (fp32 below 57344) as kParts words of four E5M2 numbers:
// three for the weight rounded to fp16, one for what that rounded off.
__device__ __forceinline__ void split(float e0, float e1, float e2, float e3,
                                      uint32_t (&w)[kParts]) {
  __half2 a = __floats2half2_rn(e0, e1), b = __floats2half2_rn(e2, e3);
  {
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    const __half2 ra = __floats2half2_rn(e0 - fa.x, e1 - fa.y);  // exact
    const __half2 rb = __floats2half2_rn(e2 - fb.x, e3 - fb.y);
    w[3] = __byte_perm(*reinterpret_cast<const uint32_t*>(&ra),
                       *reinterpret_cast<const uint32_t*>(&rb), 0x7531);
  }
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    const uint32_t ua = *reinterpret_cast<const uint32_t*>(&a);
    const uint32_t ub = *reinterpret_cast<const uint32_t*>(&b);
    // to the nearest upper byte, ties away; the third part fits one
    if (p == 2) {
      w[p] = __byte_perm(ua, ub, 0x7531);
    } else {
      const uint32_t ta = (ua + 0x00800080u) & 0xff00ff00u;
      const uint32_t tb = (ub + 0x00800080u) & 0xff00ff00u;
      w[p] = __byte_perm(ta, tb, 0x7531);
      a = __hsub2(a, *reinterpret_cast<const __half2*>(&ta));  // exact
      b = __hsub2(b, *reinterpret_cast<const __half2*>(&tb));
    }
  }
}

template <int N>
__global__ void __launch_bounds__(Plan<N>::kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ PagedAttnArgs a,
                         const Shape shape, float* __restrict__ part) {
  using PL = Plan<N>;
  constexpr int HR = PL::kRowsOf;  // rows of a softmax warp
  constexpr int kSoftWarps = 4 * PL::kGroups;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sk = base;
  uint8_t* sv = sk + PL::K * kUnitBytes;
  uint8_t* sq = sv + PL::V * kUnitBytes;   // [2][N][128]
  uint8_t* sp = sq + PL::Q;                // [2][kParts][N / 16][128][16]
  Meta& m = *reinterpret_cast<Meta*>(sp + PL::P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &m.abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&m.kfull[i], 1);
      tc::mbar_init(&m.kempty[i], 1);
      tc::mbar_init(&m.vfull[i], 1);
      tc::mbar_init(&m.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&m.sfull[i], 2);
      tc::mbar_init(&m.pfull[i], kSoftWarps);
      tc::mbar_init(&m.qfull[i], 2);
      tc::mbar_init(&m.qempty[i], kSoftWarps);
    }
    tc::mbar_init(&m.qfree, 1);
    tc::mbar_init(&m.drain, 1);
    m.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&m.tmem, PL::kCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch_map(&map_k);
    tc::tma_prefetch_map(&map_v);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = m.tmem;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    pdl_wait();
    pdl_trigger();
    Walk w;
    {
      bool bad = false;
      walk_start(a, shape, blockIdx.x, gridDim.x, w, &bad);
      if (bad && blockIdx.x == 0) raise_error(a.err, kErrBadIndex);
      if (lane == 0)
        reinterpret_cast<Cut*>(part + part_words(gridDim.x, N))[blockIdx.x] =
            cut_at(a, shape, w, blockIdx.x);
    }
    Part p;
    const int pt = kTile / a.page;         // pages of a tile
    const int oob = a.num_pages * a.Hkv * a.page;  // a row past the pool
    const uint32_t box = (uint32_t)a.page * 128;
    const float c = a.scale * kLog2e;
    Ring<PL::K> rk;
    Ring<PL::V> rv;
    int nk = 0, nv = 0;                    // copies issued, up to the stages
    bool ok = true;
    while (ok && walk_next(a, shape, w, p)) {
      const int pages = (p.l.n + a.page - 1) / a.page;
      // page ids two chunks of 32 ahead, their scales one ahead
      int at = p.t0 * pt;                  // first page of the chunk
      auto load_id = [&](int first) {
        const int pg = first + lane;
        return pg < pages && pg < p.t1 * pt
                   ? a.table[(size_t)p.b * a.max_pages + pg]
                   : -1;
      };
      int id = load_id(at), id1 = load_id(at + 32), id2 = load_id(at + 64);
      auto load_scale = [&](const float* s, int pid) {
        return pid >= 0 && pid < a.num_pages
                   ? s[(size_t)pid * a.Hkv + p.hk]
                   : 1.f;
      };
      float top_lv = -INFINITY;            // of the pages so far
      float ks = load_scale(a.k_scale, id), vs = load_scale(a.v_scale, id);
      float ks1 = load_scale(a.k_scale, id1), vs1 = load_scale(a.v_scale, id1);
      for (int t = p.t0; t < p.t1; ++t) {
        if (t * pt - at == 32) {
          at += 32;
          id = id1; ks = ks1; vs = vs1;
          id1 = id2;
          ks1 = load_scale(a.k_scale, id1);
          vs1 = load_scale(a.v_scale, id1);
          id2 = load_id(at + 64);
        }
        const int from = t * pt - at + lane;  // lane < pt: its page
        const int pid = __shfl_sync(0xffffffffu, id, from & 31);
        const bool have = lane < pt && t * pt + lane < pages;
        const bool bad = have && (pid < 0 || pid >= a.num_pages);
        if (bad) raise_error(a.err, kErrBadIndex);
        const int row = bad ? oob : (pid * a.Hkv + p.hk) * a.page;
        const uint32_t bytes = box * __popc(__ballot_sync(0xffffffffu, have));
        ok = wait_for<true>(&m.kempty[rk.at], rk.phase ^ 1, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&m.kfull[rk.at], bytes);
        __syncwarp();
        if (have)
          tc::tma_load_2d(sk + rk.at * kUnitBytes + lane * box, &map_k,
                          &m.kfull[rk.at], 0, row);
        rk.next();
        nk = min(nk + 1, PL::K);
        ok = wait_for<true>(&m.vempty[rv.at], rv.phase ^ 1, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // the copy first: the scales may still be on their way here
        if (lane == 0) expect_tx(&m.vfull[rv.at], bytes);
        __syncwarp();
        if (have)
          tc::tma_load_2d(sv + rv.at * kUnitBytes + lane * box, &map_v,
                          &m.vfull[rv.at], 0, row);
        const float pk = __shfl_sync(0xffffffffu, ks, from & 31);
        const float pv = __shfl_sync(0xffffffffu, vs, from & 31);
        const float lv = fminf(fmaxf(log2f(pv), kLeastLv), kMostLv);
        top_lv = fmaxf(top_lv, warp_top(have ? lv : -INFINITY));
        if (lane < pt) {
          m.ct[rv.at][lane] = have && !bad ? pk * c : 0.f;
          m.lv[rv.at][lane] = have ? lv : 0.f;
          m.fl[rv.at][lane] =
              lv < top_lv - kFarLv ? 0.f : tc::ex2_approx(kSumRef - lv);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.vfull[rv.at]);
        rv.next();
        nv = min(nv + 1, PL::V);
      }
    }
    // no copy is in flight when the CTA leaves, whatever the others did
    int never = 0;
    for (; nk > 0; --nk) {
      const Ring<PL::K> r = rk.back(nk);
      wait_for(&m.kfull[r.at], r.phase, &never, kWaitLimitNs);
    }
    for (; nv > 0; --nv) {
      const Ring<PL::V> r = rv.back(nv);
      wait_for(&m.vfull[r.at], r.phase, &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    // The whole warp waits, one elected thread issues: operands stay in
    // uniform registers (issued by a lone lane, an MMA cost 90 cycles).
    constexpr uint32_t id_s = tc::idesc_e4m3_f32(128, PL::kScore);
    // (of q's second part on the same columns: format 1, as in idesc_mn)
    constexpr uint32_t id_rest = id_s | (1u << 10);
    constexpr uint32_t id_o = idesc_mn(PL::kAcc);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    pdl_wait();
    pdl_trigger();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      ok = ok && wait_for(bar, par, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    Ring<PL::K> rk;
    Ring<PL::V> rv, rvs;                   // of the second, first product
    Ring<2> rs, rp;                        // scores, weights
    for (int s = 0; ok; ++s) {
      const int qb = s & 1;
      if (!wait(&m.qfull[qb], (s >> 1) & 1)) break;
      const Segment& g = m.seg[qb];
      if (g.done) break;
      const int T = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
      // The columns that tile t's scores go to were read by the softmax
      // before it handed over the weights of tile t - 2, which the second
      // product has waited for.  The softmax reads the tile's scales, which
      // came with its copy: it acquires them through the arrival below.
      auto scores = [&] {
        if (!wait(&m.kfull[rk.at], rk.phase)) return;
        if (!wait(&m.vfull[rvs.at], rvs.phase)) return;
        tc::fence_after_sync();
        const uint64_t dk =
            tc::sdesc_k_sw128(tc::smem_u32(sk) + rk.at * kUnitBytes);
        const uint64_t dq = tc::sdesc_k_sw128(tc::smem_u32(sq));
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < 2 * N / PL::kScore; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_e4m3(tm + rs.at * PL::kScore, dk + 2 * k,
                           dq + h * (N * 8) + 2 * k, h ? id_rest : id_s,
                           (h | k) != 0);
          tc::mma_commit(&m.kempty[rk.at]);
          tc::mma_commit(&m.sfull[rs.at]);
          tc::mbar_arrive(&m.sfull[rs.at]);
        }
        __syncwarp();
        rk.next();
        rvs.next();
        rs.next();
      };
      if (T > 0) scores();
      for (int t = 0; ok && t < T; ++t) {
        if (t + 1 < T) {
          scores();
        } else {                           // q is not read any more
          if (elect_one()) tc::mma_commit(&m.qfree);
          __syncwarp();
        }
        if (!wait(&m.pfull[rp.at], rp.phase)) break;
        tc::fence_after_sync();
        const uint64_t dv =
            sdesc_mn_sw128(tc::smem_u32(sv) + rv.at * kUnitBytes);
        const uint64_t dp =
            sdesc_mn_plain(tc::smem_u32(sp) + rp.at * kParts * N * 128);
        if (elect_one()) {
          // all parts side by side, or 0 and 1, then 2 and 3 onto the same
          // columns
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_e4m3(tm + 2 * PL::kScore, dv + 256 * k, dp + 32 * k, id_o,
                         t > 0 || k > 0);
          if constexpr (PL::kAcc < kParts * N) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_e4m3(tm + 2 * PL::kScore, dv + 256 * k,
                           dp + N * 16 + 32 * k, id_o, 1);
          }
          tc::mma_commit(&m.vempty[rv.at]);
        }
        __syncwarp();
        rv.next();
        rp.next();
      }
      if (T == 0) {
        if (elect_one()) tc::mma_commit(&m.qfree);
        __syncwarp();
      }
    }
    if (elect_one()) tc::mma_commit(&m.drain);
    __syncwarp();
    int never = 0;
    wait_for(&m.drain, 0, &never, kWaitLimitNs);
  } else if (warp < 4) {
    // ------------------------------------------------------ layout of q
    pdl_wait();
    pdl_trigger();
    Walk w;
    {
      bool bad = false;
      walk_start(a, shape, blockIdx.x, gridDim.x, w, &bad);
    }
    // row / g for the rows of a tile, x < kMaxRows + 64, exactly
    const uint32_t by_g = (65536 + shape.g - 1) / shape.g;
    const int qt = tid - 64;               // 0..63
    const int ch = qt & 7;                 // 16 dimensions of a row
    for (int s = 0;; ++s) {
      const int qb = s & 1;
      bool ok = wait_for<true>(&m.qempty[qb], (uint32_t)((s >> 1) & 1) ^ 1,
                               abort, a.wait_ns);
      if (s > 0)
        ok = ok && wait_for<true>(&m.qfree, (uint32_t)(s - 1) & 1, abort,
                                  a.wait_ns);
      if (any_of<64>(kQBar, !ok)) break;
      Segment& g = m.seg[qb];
      Part p;
      const bool more = walk_next(a, shape, w, p);
      if (more) {
        const int row0 = p.rt * N;
        const int q_first = row0 / shape.g, q_rest = row0 - q_first * shape.g;
        // All rows' values fly at once, asynchronously, into the place their
        // codes will take: the first 64 dimensions of a row where its upper
        // parts go, the rest where its lower parts go.  A thread reads only
        // what it copied itself.
        constexpr int J = N / 8;             // rows of a thread
        auto raw = [&](int r) {              // this thread's 32 bytes
          return sq + (ch >> 2) * N * 128 + r * 128 + (ch & 3) * 32;
        };
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
          const int r = (qt >> 3) + 8 * j, row = row0 + r;
          const int dq = (int)((uint32_t)(q_rest + r) * by_g >> 16);
          const int qi = q_first + dq;
          const int out = row < shape.rows
                              ? (p.b * a.Q + qi) * a.Hq + p.hk * shape.g +
                                    (q_rest + r - dq * shape.g)
                              : -1;
          const bool live = row < shape.rows && qi < p.l.nq;
          const bool read = live && ch * 16 < a.D;
          const uint8_t* src =
              static_cast<const uint8_t*>(a.q) +
              (read ? ((size_t)out * a.D + ch * 16) * 2 : 0);
          const uint32_t dst = tc::smem_u32(raw(r));
          copy16(dst, src, read);
          copy16(dst + 16, src + 16, read);
          if (ch == 0) {
            g.lim[r] = !live      ? 0x7fffffff
                       : a.causal ? min(p.l.n, p.l.n - p.l.nq + qi + 1)
                                  : p.l.n;
            g.out_row[r] = out;
            g.on[r] = live;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        auto fetch = [&](int r, uint32_t (&v)[8]) {
          const uint4 u0 = *reinterpret_cast<const uint4*>(raw(r));
          const uint4 u1 = *reinterpret_cast<const uint4*>(raw(r) + 16);
          v[0] = u0.x; v[1] = u0.y; v[2] = u0.z; v[3] = u0.w;
          v[4] = u1.x; v[5] = u1.y; v[6] = u1.z; v[7] = u1.w;
          float t = 0.f;                     // infinite: a NaN
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x0 = __uint_as_float(v[k] << 16);
            const float x1 = __uint_as_float(v[k] & 0xffff0000u);
            t = x0 == x0 ? fmaxf(t, fabsf(x0)) : INFINITY;
            t = x1 == x1 ? fmaxf(t, fabsf(x1)) : INFINITY;
          }
#pragma unroll
          for (int o = 4; o; o >>= 1)
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
          return t;                          // the row's largest value
        };
        float all = 0.f;
#pragma unroll 2
        for (int j = 0; j < J; ++j) {
          uint32_t v[8];
          const float t = fetch((qt >> 3) + 8 * j, v);
          if (t < INFINITY) all = fmaxf(all, t);
        }
        all = warp_max(all);
        if (lane == 0) m.q_top[warp - 2] = all;
        any_of<64>(kQBar, false);
        all = fmaxf(m.q_top[0], m.q_top[1]);
        // the unit's largest value to [128, 256)
        const int e_all = max((int)(__float_as_uint(all) >> 23) - 127, -100);
        bool own = false;
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
          const int r = (qt >> 3) + 8 * j;
          uint32_t v[8];
          const float big = fetch(r, v);  // the whole row has been read now
          const int e_row = (int)(__float_as_uint(big) >> 23) - 127;
          int e = e_all;
          if (big > 0.f && e_row < e_all - kRowsApart) {
            e = max(e_row, max(-100, e_all - 100));
            own = true;
          }
          const float up = big < INFINITY
                               ? __uint_as_float((134 - e) << 23)
                               : __uint_as_float(0x7fffffffu);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 y =
                make_float2(__uint_as_float(v[k] << 16) * up,
                            __uint_as_float(v[k] & 0xffff0000u) * up);
            const uint32_t h =
                __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            const float2 f = __half22float2(
                __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
            const float2 rest = make_float2((y.x - f.x) * PL::kRestUp,
                                            (y.y - f.y) * PL::kRestUp);
            const uint32_t l =
                __nv_cvt_float2_to_fp8x2(rest, __NV_SATFINITE, PL::kRestType);
            if (k & 1) {
              hi[k >> 1] |= h << 16;
              lo[k >> 1] |= l << 16;
            } else {
              hi[k >> 1] = h;
              lo[k >> 1] = l;
            }
          }
          uint8_t* dst = sq + r * 128 + ((ch ^ (r & 7)) << 4);
          __syncwarp();
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + N * 128) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (ch == 0) g.rel[r] = __uint_as_float((127 + e - e_all) << 23);
        }
        own = any_of<64>(kQBar, own);
        if (qt == 0) {
          g.uneven = own;
          g.back = __uint_as_float((120 + e_all) << 23);  // 2^(e_all - 7)
        }
        if (qt == 0) {
          g.b = p.b;
          g.hk = p.hk;
          g.row0 = row0;
          g.t0 = p.t0;
          g.t1 = p.t1;
          g.n = p.l.n;
          g.nq = p.l.nq;
          g.whole = p.whole;
          g.slot = 2 * blockIdx.x + (p.first ? 0 : 1);
          g.min_lim =
              a.causal ? min(p.l.n, p.l.n - p.l.nq + q_first + 1) : p.l.n;
        }
      }
      if (qt == 0) g.done = !more;
      fence_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&m.qfull[qb]);
      if (!more) break;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int half = (warp - 4) >> 2, quarter = warp & 3;  // half: the group
    const int ht = tid - 128 - half * 128;  // thread of the group
    const int tok = quarter * 32 + lane;
    const int bar = 1 + half;
    // Row `row_of(r)` of the unit is row r (a multiple of 4) of the group.  A
    // group holds whole units of 16 rows, whose bytes one store writes; the
    // rest of the groups' rows share the last units.
    constexpr int kFull = HR / 16 * 16, kRest = HR - kFull;
    static_assert(PL::kGroups * kRest % 16 == 0 && kRest % 4 == 0, "");
    auto row_of = [&](int r) {
      return r < kFull ? half * kFull + r
                       : PL::kGroups * kFull + half * kRest + r - kFull;
    };
    // The same as offsets from the group's first and first shared row.
    const int full0 = half * kFull, rest0 = PL::kGroups * kFull + half * kRest;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    auto col_of = [&](uint32_t base, int r) {
      return r < kFull ? base + full0 + r : base + rest0 + (r - kFull);
    };
    const uint32_t o_col = lanes + 2 * PL::kScore;
    const float* ref_full = m.neg_ref + full0;
    const float* ref_rest = m.neg_ref + rest0;
    uint8_t* p_full = sp + tok * 16 + full0 * 128;  // 2048 bytes to 16 rows
    uint8_t* p_rest = sp + tok * 16 + (rest0 >> 4) * 2048 + (rest0 & 12);
    const int my_row = ht < HR ? row_of(ht & ~3) + (ht & 3) : 0;
    constexpr int SG = PL::kScore / N;     // columns of a row's score
    constexpr int OG = PL::kAcc / N;       // and of its accumulator
    const int page_bits = __ffs(a.page) - 1;
    Ring<2> rs;
    Ring<PL::V> rv;
    bool live = true;
    // s = -1: one tile of a segment that is not there.  It waits for nothing,
    // signals nothing and writes nothing that is read, but brings the code of
    // the tile, of the raised reference and of the output (first executions
    // of which took 6000 to 10000 cycles) into the instruction caches while
    // the lengths, q and the first tile are on their way.
    for (int s = -1; live; ++s) {
      const bool dry = s < 0;
      const int qb = s & 1;
      if (s == 0) {  // the outputs may still be read by the launch before
        pdl_wait();
        pdl_trigger();
      }
      bool ok = dry || wait_for(&m.qfull[qb], (s >> 1) & 1, abort, a.wait_ns);
      if (half_any(bar, !ok)) break;
      const Segment& g = m.seg[qb];
      if (!dry && g.done) break;
      const int T = dry ? 1 : g.t1 - g.t0, n = dry ? 0x7fffffff : g.n;
      // tokens from the segment's start
      const int mask_from = dry ? 0x7fffffff : g.min_lim - g.t0 * kTile;
      const bool uneven = !dry && g.uneven;
      const bool whole = dry || g.whole;
      const float back = dry ? 0.f : g.back;
      int pos = dry ? tok : g.t0 * kTile + tok;  // this thread's token
      uint64_t l[HR / 2];   // sums of weights, by pairs of rows
#pragma unroll
      for (int r = 0; r < HR / 2; ++r) l[r] = 0;
      // kHead - reference; 0 before the first tile
      if (ht < HR) m.neg_ref[my_row] = 0.f;
      half_sync(bar);
      // The scores of buffer `at` into y: asked for by ask(), there after
      // got().  With more than 32 rows the softmax sets the pace, and the
      // next tile's scores, if ready, are asked for while this tile's weights
      // are handed over: 36 rows 78 -> 74 us, 72 rows 99 -> 96 us (eight
      // sequences of 16,384); with fewer the cache does, and one row of
      // 131,072 tokens went from 58 to 60 us.
      float y[HR], z[SG == 2 ? HR : 1];
      auto ask = [&](int at) {
        tc::fence_after_sync();
        const uint32_t s_col = lanes + at * PL::kScore;
#pragma unroll
        for (int r = 0; r < HR; r += 4) tmem_ld4(col_of(s_col, r), y + r);
        if constexpr (SG == 2) {
#pragma unroll
          for (int r = 0; r < HR; r += 4) tmem_ld4(col_of(s_col + N, r), z + r);
        }
      };
      auto got = [&] {
        if constexpr (SG == 2) {
          tmem_loaded(z);
          tmem_loaded(y);
#pragma unroll
          for (int r = 0; r < HR; r += 2)
            unpack2(fma2(pack2(z[r], z[r + 1]),
                         pack2(1.f / PL::kRestUp, 1.f / PL::kRestUp),
                         pack2(y[r], y[r + 1])), y[r], y[r + 1]);
        } else {
          tmem_loaded(y);
        }
        tc::fence_before_sync();
      };
      bool early = false;  // y holds this tile's scores already
      for (int t = 0; t < T; ++t, pos += kTile) {
        const int sb = rs.at, st = rv.at;
        // Also says that the weights' buffer is free: the scores' commit
        // follows the second product of two tiles ago.
        if (!early) {
          ok = dry || wait_for(&m.sfull[sb], rs.phase, abort, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            ask(sb);
            got();
          } else {
#pragma unroll
            for (int r = 0; r < HR; ++r) y[r] = 0.f;
          }
        }
        const int pg = tok >> page_bits;
        const float ct = m.ct[st][pg] * back, lv = m.lv[st][pg];
        const float fl = m.fl[st][pg];
        if (uneven) {
#pragma unroll
          for (int r = 0; r < HR; ++r) y[r] *= g.rel[row_of(r & ~3) + (r & 3)];
        }
        const uint64_t ct2 = pack2(ct, ct), lv2 = pack2(lv, lv);
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          const ulonglong2 nr =
              *reinterpret_cast<const ulonglong2*>(
                  r < kFull ? ref_full + r : ref_rest + (r - kFull));
          unpack2(add2(fma2(pack2(y[r], y[r + 1]), ct2, lv2), nr.x), y[r],
                  y[r + 1]);
          unpack2(add2(fma2(pack2(y[r + 2], y[r + 3]), ct2, lv2), nr.y),
                  y[r + 2], y[r + 3]);
        }
        if ((t + 1) * kTile > mask_from) {
#pragma unroll
          for (int r = 0; r < HR; ++r)
            y[r] = pos < min(g.lim[row_of(r & ~3) + (r & 3)], n) ? y[r]
                                                               : -INFINITY;
        }
        float top = fmaxf(y[0], y[1]);
#pragma unroll
        for (int r = 2; r < HR; r += 2) top = fmaxf(fmaxf(y[r], y[r + 1]), top);
        if (half_any(bar, t == 0 || top > kRaise || !ok)) {
          // ---- raise the references -------------------------------------
          if (half_any(bar, !ok)) { live = false; break; }
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            const float z = warp_top(y[r]);
            if (lane == 0) m.warp_val[quarter][row_of(r & ~3) + (r & 3)] = z;
          }
          half_sync(bar);
          if (ht < HR) {
            const int r = my_row;
            const float z =
                fmaxf(fmaxf(m.warp_val[0][r], m.warp_val[1][r]),
                      fmaxf(m.warp_val[2][r], m.warp_val[3][r]));
            // nothing to raise for a row that sees nothing yet
            const float d = z > -INFINITY && (t == 0 || z > kHead)
                                ? kHead - ceilf(z) : 0.f;
            m.fac[r] = d;
            m.neg_ref[r] += d;
          }
          half_sync(bar);
          if (t > 0) {
            const Ring<PL::V> before = rv.back(1);
            ok = wait_for(&m.vempty[before.at], before.phase, abort, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
          }
#pragma unroll
          for (int r = 0; r < HR; r += 4) {
            const float4 d =
                *reinterpret_cast<const float4*>(&m.fac[row_of(r)]);
            // In two factors: the sums may hold what the weights do not.  A
            // reference falls only in the first tile, where there is nothing
            // to scale yet (2^d may pass fp32's range).
            const float e[4] = {d.x, d.y, d.z, d.w};
            float f[4], f2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[r + k] += e[k];
              f[k] = tc::ex2_approx(fminf(fmaxf(e[k], -100.f), 0.f));
              f2[k] = tc::ex2_approx(fminf(e[k] + 100.f, 0.f));
            }
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              uint64_t& lr = l[(r + k) / 2];
              lr = mul2(mul2(lr, pack2(f[k], f[k + 1])),
                        pack2(f2[k], f2[k + 1]));
            }
            const bool one = d.x == 0.f && d.y == 0.f && d.z == 0.f &&
                             d.w == 0.f;
            if (t > 0 && !one && ok) {
#pragma unroll
              for (int h = 0; h < OG; ++h) {
                float o[4];
                tmem_ld4(o_col + h * N + row_of(r), o);
                tmem_loaded(o);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] *= f[k] * f2[k];
                tmem_st4(o_col + h * N + row_of(r), o);
              }
            }
          }
          if (t > 0) {
            tmem_stored();
            tc::fence_before_sync();
          }
        }
        if (fl == 0.f) {
#pragma unroll
          for (int r = 0; r < HR; r += 2)
            l[r / 2] = add2(l[r / 2],
                            pack2(tc::ex2_approx(y[r] + (kSumRef - lv)),
                                  tc::ex2_approx(y[r + 1] + (kSumRef - lv))));
        }
        // ---- the weights, in parts -----------------------------------------
        const int p_buf = sb * kParts * N * 128;
        const uint64_t fl2 = pack2(fl, fl);
#pragma unroll
        for (int r = 0; r < HR; r += 16) {
          const int words = HR - r < 16 ? kRest / 4 : 4;  // of four rows
          uint32_t c[4][kParts];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= words) break;
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              e[j] = tc::ex2_approx(y[r + 4 * k + j]);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              uint64_t& lr = l[(r + 4 * k + j) / 2];
              lr = fma2(pack2(e[j], e[j + 1]), fl2, lr);
            }
            split(e[0], e[1], e[2], e[3], c[k]);
          }
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            uint8_t* at =
                (r < kFull ? p_full + r * 128 : p_rest) + p_buf + h * N * 128;
            if (words == 4)
              *reinterpret_cast<uint4*>(at) =
                  make_uint4(c[0][h], c[1][h], c[2][h], c[3][h]);
            else if (words == 2)
              *reinterpret_cast<uint2*>(at) = make_uint2(c[0][h], c[1][h]);
            else
              *reinterpret_cast<uint32_t*>(at) = c[0][h];
          }
        }
        if (half == 0 && pos >= n && ok) {
          // values past the cache's end may be anything: their weight is 0
          uint4* v = reinterpret_cast<uint4*>(sv + st * kUnitBytes + tok * 128);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = make_uint4(0, 0, 0, 0);
        }
        early = false;
        if (!dry) {
          rs.next();
          rv.next();
          if (N > 32 && t + 1 < T)
            early = tc::mbar_try_wait(&m.sfull[rs.at], rs.phase, 0);
        }
        early = __all_sync(0xffffffffu, early);
        // No branch between ask() and got(): the registers are in flight.
        if (early) {
          ask(rs.at);
          fence_async();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.pfull[sb]);
          got();
        } else {
          fence_async();
          __syncwarp();
          if (!dry && lane == 0) tc::mbar_arrive(&m.pfull[sb]);
        }
      }
      if (!live) break;
      // ---- the segment's result ------------------------------------------
      if (T > 0) {
        const Ring<PL::V> last = rv.back(1);
        ok = dry || wait_for(&m.vempty[last.at], last.phase, abort, a.wait_ns);
        if (half_any(bar, !ok)) break;
        tc::fence_after_sync();
      }
      {
        float v[HR];
#pragma unroll
        for (int r = 0; r < HR; r += 2) unpack2(l[r / 2], v[r], v[r + 1]);
        int from = 0;
        lane_sums<HR, 16>(v, lane, from);
#pragma unroll
        for (int i = 0; i < lane_share(HR, 16); ++i) {
          const int r = from + i;  // some lanes hold the same sums
          m.warp_val[quarter][row_of(r & ~3) + (r & 3)] = v[i];
        }
      }
      half_sync(bar);
      if (ht < HR) {
        const int r = my_row;
        const float sum = (m.warp_val[0][r] + m.warp_val[1][r]) +
                          (m.warp_val[2][r] + m.warp_val[3][r]);
        const bool seen = sum > 0.f || sum != sum;  // a NaN stays one
        // sum = frac 2^ex; 2^ref: what frac counts.  (Parts of runs whose
        // value scales lie far apart join by that.)
        const int ex =
            min(max((int)(__float_as_uint(sum) >> 23) - 127, -100), 120);
        const float frac = sum * __uint_as_float((127 - ex) << 23);
        const float ref = (float)ex - m.neg_ref[r] - kSumRef;
        if (whole) {
          const bool on = seen && g.on[r];
          m.fac[r] = on ? exp2f(kSumRef) / sum : 0.f;
          if (!dry && g.out_row[r] >= 0 && a.lse)
            a.lse[g.out_row[r]] =
                on ? (log2f(frac) + ref) * 0.6931471805599453f : -INFINITY;
        } else {
          m.fac[r] = __uint_as_float((127 + (int)kSumRef - ex) << 23);
          float2* ml = reinterpret_cast<float2*>(
              part + (size_t)2 * gridDim.x * N * 128);
          ml[(size_t)g.slot * N + r] =
              make_float2(seen ? ref : -INFINITY, seen ? frac : 0.f);
        }
      }
      half_sync(bar);
      const int d = tok;
#pragma unroll
      for (int r = 0; r < HR; r += 4) {
        float o[4 * OG];
        if (T > 0) {
#pragma unroll
          for (int h = 0; h < OG; ++h)
            tmem_ld4(o_col + h * N + row_of(r), o + 4 * h);
          tmem_loaded(o);
        } else {
#pragma unroll
          for (int k = 0; k < 4 * OG; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = row_of(r) + k;
          const float f = m.fac[row];
          float v = o[k];
#pragma unroll
          for (int h = 1; h < OG; ++h) v += o[4 * h + k];
          v *= f;
          if (whole) {
            const int at = dry ? -1 : g.out_row[row];
            if (at >= 0 && d < a.D)
              static_cast<__nv_bfloat16*>(a.out)[(size_t)at * a.D + d] =
                  __float2bfloat16_rn(f == 0.f ? 0.f : v);
          } else {
            part[((size_t)g.slot * N + row) * 128 + d] = v;
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (!dry && lane == 0) tc::mbar_arrive(&m.qempty[qb]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, PL::kCols);
  if (tid == 0 && m.abort) raise_error(a.err, kErrTimeout);
}

// Joins the partial sums of the units that the runs cut: a CTA for each that
// may have left one, a warp per row, eight rows of the unit to a CTA.  (With a
// CTA for every unit that counted the work before it, the join took 27 ms of
// 30 for a prompt of 8192 tokens and 64 heads.)
constexpr int kJoinRows = 8;
constexpr int kJoinThreads = 32 * kJoinRows;
__global__ void __launch_bounds__(kJoinThreads)
    paged_attn_tc_join_kernel(const __grid_constant__ PagedAttnArgs a,
                              const Shape shape, int grid,
                              const float* __restrict__ part) {
  __shared__ float s_w[kJoinRows][kMaxCtas];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  const int cta = blockIdx.x + 1;
  const Cut cut =
      reinterpret_cast<const Cut*>(part + part_words(grid, shape.N))[cta];
  if (cut.parts == 0) return;
  const int r = blockIdx.y * kJoinRows + warp;
  const int row = cut.rt * shape.N + r;
  if (r >= shape.N || row >= shape.rows) return;
  const int n = cut.parts >> 1, odd = cut.parts & 1, c0 = cta - 1;
  const int b = cut.b, hk = cut.hk;
  auto slot = [&](int i) { return 2 * (c0 + i) + (i == 0 ? odd : 0); };
  const float2* ml = reinterpret_cast<const float2*>(
      part + (size_t)2 * grid * shape.N * 128);
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32)
    top = fmaxf(top, ml[(size_t)slot(i) * shape.N + r].x);
  top = warp_max(top);
  float sum = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float2 v = ml[(size_t)slot(i) * shape.N + r];
    const float w = v.x == -INFINITY ? 0.f : exp2f(v.x - top);
    s_w[warp][i] = w;
    sum += w * v.y;
  }
  sum = warp_sum(sum);
  __syncwarp();
  const int qi = row / shape.g;
  const size_t at =
      ((size_t)b * a.Q + qi) * a.Hq + hk * shape.g + row % shape.g;
  bool bad = false;
  const bool on =
      (sum > 0.f || sum != sum) && qi < lens_of(a, b, &bad).nq;
  const float inv = on ? 1.f / sum : 0.f;
  if (lane == 0 && a.lse)
    a.lse[at] = on ? (log2f(sum) + top) * 0.6931471805599453f : -INFINITY;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float w = s_w[warp][i];
    const float4 v = *reinterpret_cast<const float4*>(
        part + ((size_t)slot(i) * shape.N + r) * 128 + 4 * lane);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  if (4 * lane < a.D) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    uint2 v;
    v.x = *reinterpret_cast<const uint32_t*>(&x);
    v.y = *reinterpret_cast<const uint32_t*>(&y);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                              at * a.D + 4 * lane) = v;
  }
}

Shape shape_of(long long Q, int Hq, int Hkv) {
  Shape s;
  s.g = Hq / Hkv;
  s.rows = (int)(Q * s.g);
  s.row_tiles = (s.rows + kMaxRows - 1) / kMaxRows;
  const int per = (s.rows + s.row_tiles - 1) / s.row_tiles;
  s.N = (per + 15) / 16 * 16;
  s.row_tiles = (s.rows + s.N - 1) / s.N;
  return s;
}

template <int N>
cudaError_t launch_n(const CUtensorMap& mk, const CUtensorMap& mv,
                     const PagedAttnArgs& a, const Shape& s, int G,
                     float* part, cudaStream_t stream) {
  auto* f = paged_attn_tc_kernel<N>;
  cudaError_t e = cudaFuncSetAttribute(
      f, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<N>::kBytes);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(G), dim3(Plan<N>::kThreads), Plan<N>::kBytes, stream);
  return cudaLaunchKernelEx(&L.cfg, f, mk, mv, a, s, part);
}

}  // namespace

bool paged_attn_tc_takes(int D, dflash_dtype dt) {
  return dt == DFLASH_BF16 && D <= 128;
}

size_t paged_attn_tc_ws(int B, int Q, int Hq, int Hkv) {
  (void)B;
  const Shape s = shape_of(Q, Hq, Hkv);
  return part_words(kMaxCtas, s.N) * sizeof(float) + kMaxCtas * sizeof(Cut);
}

cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, int sms, float* part,
                                 cudaStream_t stream) {
  const Shape s = shape_of(a.Q, a.Hq, a.Hkv);
  const long long most =
      (long long)a.B * a.Hkv * s.row_tiles *
      (((long long)a.max_pages * a.page + kTile - 1) / kTile + kUnitCost);
  if (most > 0x7fffffffll) return cudaErrorNotSupported;
  const int G = std::min(sms, kMaxCtas);
  CUtensorMap mk, mv;
  const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * a.page;
  if (!make_tmap_u8_2d(&mk, a.k_codes, a.D, rows, 128, a.page) ||
      !make_tmap_u8_2d(&mv, a.v_codes, a.D, rows, 128, a.page))
    return cudaErrorInvalidValue;
  cudaError_t e;
  switch (s.N) {
    case 16: e = launch_n<16>(mk, mv, a, s, G, part, stream); break;
    case 32: e = launch_n<32>(mk, mv, a, s, G, part, stream); break;
    case 48: e = launch_n<48>(mk, mv, a, s, G, part, stream); break;
    case 64: e = launch_n<64>(mk, mv, a, s, G, part, stream); break;
    case 80: e = launch_n<80>(mk, mv, a, s, G, part, stream); break;
    default: e = launch_n<96>(mk, mv, a, s, G, part, stream); break;
  }
  if (e != cudaSuccess) return e;
  if (G < 2) return e;
  const int rows_of = std::min(s.N, s.rows);
  PdlLaunch J(dim3(G - 1, (rows_of + kJoinRows - 1) / kJoinRows),
              dim3(kJoinThreads), 0, stream);
  return cudaLaunchKernelEx(&J.cfg, paged_attn_tc_join_kernel, a, s, G,
                            (const float*)part);
}

}  // namespace dflash
