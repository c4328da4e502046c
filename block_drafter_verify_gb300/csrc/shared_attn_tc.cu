// Attention of a batch whose sequences share their first tokens, on the tensor
// cores (tcgen05), for bf16 queries and heads of up to 128 dimensions.
//
// The rows (query, head) of all sequences that read a key head are numbered
// through.  A unit is up to 256 of them, in two halves of 128, with the tokens
// that they see: of all sequences with the shared tokens, of one sequence with
// its own.  Both are tiles of 128 tokens: S = Q K^T (a row to a TMEM lane, so a
// thread owns a row and its sums), P = weights, O += P V.
//   K and V  are taken to fp16 on their way (four warps, from the tile that TMA
//            brought to two operands as the MMA reads them): E4M3 codes are
//            exact there.  That costs the 8-bit MMA's rate, but then one product
//            does where the codes as they are need q in two and the weights in
//            four 8-bit parts, and with 128 and 256 rows to a tile the products
//            are what counts.
//   q        is scaled by a power of two for each row, its largest value to
//            [2^14, 2^15): fp16 then holds all of bf16's bits down to 2^-28 of
//            that value.
//   P        fp16: to 2^-11 of a weight, or 2^-34 of the row's largest
//            (which is 2^9 or more).  The sum counts weights as they are in
//            fp32.
// The page's scales are one factor and one addend of the exponent for 16 columns:
// weights carry their value's scale, the row's sum is taken without it (see
// kSumRef).  The running maximum is lazy: weights are taken against a reference
// that is raised (sum and accumulator rescaled, by an exact power of two) only
// when a token beats it by more than 2^5.75.
//
// All tiles of all units are numbered, and every CTA (one per SM) takes an equal
// run of them by cost.  A run's parts of units go to the workspace, and a second
// launch joins each row's: of the shared tokens and of its sequence's own.
//
// Warps: 0 copies tiles (TMA, one box per page), 1 issues the MMAs, 2 hands out
// the segments of the run, 4-7 convert, 8-15 (a group of four to a half) lay out
// q, do the softmax and write the parts.  While one half's softmax runs, the
// tensor cores have the other's products.  Every wait is bounded; on a timeout
// the CTA stops issuing, drains, frees TMEM and flags the error word.
//
// What bounds it: the chain of a half's tile (scores, their two readings by the
// softmax, weights, products) and its handshakes, 5900 cycles for 256 rows by
// 128 tokens of which the tensor pipe has 2100.  64 sequences of 9 tokens, 64
// query and 8 key heads, 16384 shared and up to 2000 own tokens: 519 us, 540
// TFLOP/s, the tensor pipe 33 %, issue slots 41 %.  Tiles of 64 tokens with two
// score buffers a half and an issuer for each: the same.  The softmax's loops
// are not unrolled and rare paths are kept short: the roles' code passes the
// instruction caches, and each step that made it shorter gained 3 to 10 %.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "attn_roles.cuh"
#include "kernels.h"

namespace dflash {
namespace {

constexpr int kTile = 128;          // tokens of a tile
constexpr int kHalf = 128;          // rows of a half
constexpr int kRows = 2 * kHalf;    // most rows of a unit
constexpr int kMaxCtas = 160;
constexpr int kThreads = 512;
constexpr int kRawBytes = kTile * 128;      // a tile of codes
constexpr int kWideBytes = 2 * kRawBytes;   // and as fp16
constexpr int kRaw = 2, kWide = 4;          // stages: K and V by turns
constexpr int kInfo = 8;                    // tiles' scales in flight
constexpr int kSegs = 4;                    // segments handed out ahead
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHead = 10.f;       // weights are 2^(score - ref + kHead)
constexpr float kRaise = 15.75f;    // 2^15.75 = 55109 < 65504
// A row's sum counts its weights without their value scales (2^lv), times
// 2^kSumRef: with scales from 2^kLeastLv to 2^kMostLv and 2^30 tokens it stays
// between 2^-95 and 2^126, whichever of them the reference has come from.
constexpr float kSumRef = 16.f;
constexpr float kLeastLv = -64.f, kMostLv = 120.f;
// Weights of pages whose value scale is that much (in bits) below the largest
// of the run so far may underflow: their terms of the sum are computed apart.
constexpr float kFarLv = 90.f;
// Work is counted in tiles of one half; a unit's start and end take kUnitCost.
constexpr int kUnitCost = 4;

// Part of a unit that a CTA works on.
struct Segment {
  int done;               // no more work
  int prefix;             // the shared tokens' (of all sequences)
  int b, hk;              // row of the page table, key head
  int row0, rows;         // rows of the head
  int tok0, T, end;       // first token, tiles, end of the tokens
  int slot;               // where the part goes; -1: the whole unit, by row
};

struct Meta {
  Segment seg[kSegs];
  // of 16 tokens: key factor, log2 of the value scale, 2^(kSumRef - that) or 0
  alignas(16) float4 info[kInfo][kTile / 16];
  uint64_t raw_full[kRaw], raw_empty[kRaw], wide_full[kWide], wide_empty[kWide];
  uint64_t s_full[2], p_full[2], q_full[2], o_full[2];
  uint64_t x_full, x_empty;
  alignas(8) float2 x[kHalf];  // the second half's sums and references
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};
constexpr int kQBytes = kRows * 128 * 2;
constexpr int kSmem = kQBytes + kWide * kWideBytes + kRaw * kRawBytes +
                      ((int)sizeof(Meta) + 15) / 16 * 16;
static_assert(kSmem <= 232448, "");

// ---- the numbering of the work ---------------------------------------------
struct Shape {
  int g;                  // query heads of a key head
  int own, all;           // rows of a head: a sequence's, all sequences'
  int own_units, all_units;
  int shared, tiles;      // shared tokens, their tiles
};
__host__ __device__ __forceinline__ int cost_of(int rows, int unit) {
  return rows - unit * kRows > kHalf ? 2 : 1;
}
__host__ __device__ __forceinline__ int work_of(int T, int cost) {
  return T > 0 ? kUnitCost + T * cost : 0;
}
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
// Own tokens' tiles of unit u of a sequence.
__device__ __forceinline__ int tiles_of(const PagedAttnArgs& a, const Shape& s,
                                        const Lens& l, int u) {
  const int q0 = u * kRows / s.g;
  if (q0 >= l.nq) return 0;
  int seen = l.n;
  if (a.causal) {
    const int q1 = min((min((u + 1) * kRows, s.own) - 1) / s.g, l.nq - 1);
    seen = max(0, min(l.n, l.n - l.nq + q1 + 1));
  }
  return (max(0, seen - s.shared) + kTile - 1) / kTile;
}
// Work of one key head: the shared tokens', a sequence's own.
__host__ __device__ __forceinline__ int shared_work(const Shape& s) {
  return (s.all_units - 1) * work_of(s.tiles, 2) +
         work_of(s.tiles, cost_of(s.all, s.all_units - 1));
}
__device__ __forceinline__ int own_work(const PagedAttnArgs& a, const Shape& s,
                                        const Lens& l) {
  int w = 0;
#pragma unroll 1
  for (int u = 0; u < s.own_units; ++u)
    w += work_of(tiles_of(a, s, l, u), cost_of(s.own, u));
  return w;
}
// First position of CTA c of the G that work, which have `total` = q G + r.
struct Runs {
  int q, r, G;
  __device__ __forceinline__ int start(int c) const {
    return q * c + r * c / G;
  }
};
// Tiles of a unit before position `at` of it.
__device__ __forceinline__ int tiles_before(int at, int T, int cost) {
  return at <= kUnitCost ? 0 : min(T, (at - kUnitCost + cost - 1) / cost);
}

// Walks the units from a position in the numbering.  (Calls: inlined, the walk
// took registers that the softmax needs.)
struct Walk {
  int b, hk, u, at;       // b = -1: the shared tokens; at: position in the unit
  int left;               // positions left in this CTA's run
  int pos;                // position among all
  int shared_end;         // of the shared tokens that some sequence has
  Runs runs;
};
// A unit that has tiles, as the CTA that begins it leaves it for the join: its
// first position, the first and last CTA that have some of it, its tiles.
struct alignas(16) Begun {
  int first, c0, c1, T;
};
__host__ __device__ __forceinline__ size_t unit_of(const Shape& s, int Hkv,
                                                   int b, int hk, int u) {
  return b < 0 ? (size_t)hk * s.all_units + u
               : (size_t)Hkv * s.all_units +
                     ((size_t)b * Hkv + hk) * s.own_units + u;
}
// Where the run of CTA `cta` of `grid` starts.  A whole warp, each lane with a
// stretch of the sequences; *bad: some length was out of range.
__device__ __noinline__ void walk_start(const PagedAttnArgs& a,
                                        const Shape& s, int cta, int grid,
                                        Walk& w, bool* bad) {
  const int lane = threadIdx.x & 31;
  const int per = (a.B + 31) / 32;
  const int b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
  int work = 0, longest = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Lens l = lens_of(a, b, bad);
    work += a.Hkv * own_work(a, s, l);
    longest = max(longest, l.n);
  }
  int run = work;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  const int head = shared_work(s), first = a.Hkv * head;
  run += first;
  const int total = __shfl_sync(0xffffffffu, run, 31);
  const int G = min(grid, total);
  // (what lies behind the longest sequence may be anything)
  const int shared_end =
      min(s.shared, __reduce_max_sync(0xffffffffu, longest));
  w = Walk{0, 0, 0, 0, 0, 0, shared_end, Runs{0, 0, G}};
  if (cta >= G) return;                    // the same in every lane
  w.runs.q = total / G;
  w.runs.r = total - w.runs.q * G;
  const int p0 = w.runs.start(cta);
  w.left = w.runs.start(cta + 1) - p0;
  w.pos = p0;
  if (p0 < first) {
    w.b = -1;
    w.hk = p0 / head;
    w.at = p0 - w.hk * head;
    const int full = work_of(s.tiles, 2);
    w.u = min(w.at / full, s.all_units - 1);
    w.at -= w.u * full;
    return;
  }
  const bool mine = p0 >= run - work && p0 < run;
  int o = p0 - (run - work);
  if (mine) {
    int h = 1;
#pragma unroll 1
    for (w.b = b0; w.b < b1; ++w.b) {
      h = own_work(a, s, lens_of(a, w.b, bad));
      if (o < a.Hkv * h) break;
      o -= a.Hkv * h;
    }
    w.hk = o / h;
    o -= w.hk * h;
    const Lens l = lens_of(a, w.b, bad);
#pragma unroll 1
    for (;; ++w.u) {
      const int t = work_of(tiles_of(a, s, l, w.u), cost_of(s.own, w.u));
      if (o < t) break;
      o -= t;
    }
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  w.b = __shfl_sync(0xffffffffu, w.b, from);
  w.hk = __shfl_sync(0xffffffffu, w.hk, from);
  w.u = __shfl_sync(0xffffffffu, w.u, from);
  w.at = __shfl_sync(0xffffffffu, o, from);
}
// The next segment; false at the end of the run.  The units that begin in the
// run go to `begun`.
__device__ __noinline__ bool walk_next(const PagedAttnArgs& a, const Shape& s,
                                       Walk& w, int cta, Segment& g,
                                       Begun* begun) {
  bool bad = false;
  while (w.left > 0) {
    const bool prefix = w.b < 0;
    const Lens l = prefix ? Lens{0, 0} : lens_of(a, w.b, &bad);
    const int T = prefix ? s.tiles : tiles_of(a, s, l, w.u);
    const int cost = cost_of(prefix ? s.all : s.own, w.u);
    const int work = work_of(T, cost);
    const int from = w.at, end = min(work, from + w.left);
    const int t0 = tiles_before(from, T, cost), t1 = tiles_before(end, T, cost);
    const int b = w.b, hk = w.hk, u = w.u;
    if (from == 0 && T > 0 && (threadIdx.x & 31) == 0) {
      int last = cta;                       // CTA of the unit's last position
      while (w.runs.start(last + 1) < w.pos + work) ++last;
      begun[unit_of(s, a.Hkv, b, hk, u)] = Begun{w.pos, cta, last, T};
    }
    w.pos += end - from;
    w.left -= end - from;
    w.at = end;
    if (end == work) {
      w.at = 0;
      if (++w.u == (prefix ? s.all_units : s.own_units)) {
        w.u = 0;
        if (++w.hk == a.Hkv) {
          w.hk = 0;
          ++w.b;
        }
      }
    }
    if (t1 > t0) {
      const int tok = prefix ? 0 : s.shared;
      g.done = 0;
      g.prefix = prefix;
      g.b = prefix ? 0 : b;
      g.hk = hk;
      g.row0 = (prefix ? 0 : b * s.own) + u * kRows;
      g.rows = min(kRows, (prefix ? s.all : s.own) - u * kRows);
      g.tok0 = tok + t0 * kTile;
      g.T = t1 - t0;
      g.end = prefix ? w.shared_end : l.n;
      g.slot = t1 - t0 == T ? -1 : 2 * cta + (from > 0 ? 0 : 1);
      return true;
    }
  }
  g.done = 1;
  return false;
}

// ---- the workspace -----------------------------------------------------------
// Parts of rows: D sums of weights times values, and {reference, sum of
// weights}: of the runs' cut units by slot, then of whole units by row (index
// of out's row), of the shared tokens and of the own.
struct Parts {
  float* o;
  float2* ml;
  Runs* runs;
  Begun* begun;
  size_t by_row;           // first of the parts by row
};
__host__ __device__ inline Parts parts_of(void* ws, size_t rows, int D) {
  Parts p;
  p.by_row = (size_t)2 * kMaxCtas * kRows;
  const size_t n = p.by_row + 2 * rows;
  p.o = static_cast<float*>(ws);
  p.ml = reinterpret_cast<float2*>(p.o + n * D);
  p.runs = reinterpret_cast<Runs*>(p.ml + n);       // (16 bytes)
  p.begun = reinterpret_cast<Begun*>(
      reinterpret_cast<uint8_t*>(p.runs) + 16 + (n & 1) * 8);
  return p;
}

// ---- PTX -----------------------------------------------------------------------
// kind::f16 with fp16 operands (format 0), fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(kHalf >> 4) << 24);
}
// B with N contiguous (bit 16).
__host__ __device__ constexpr uint32_t idesc_f16_mn(int N) {
  return idesc_f16(N) | (1u << 16);
}
// N contiguous in 128-byte rows (64 values of a token) with 128-byte swizzle:
// groups of eight tokens 1024 bytes apart (stride), blocks of 64 values 16 KB
// apart (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_wide(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>(kRawBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a,
                                           uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(
          d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A factor of scores: a masked one (-inf) has to stay that, so it is not 0.
__device__ __forceinline__ float factor(float f) {
  return fmaxf(f, 0x1p-126f);
}

// How a segment's tiles fall to the halves: with more than 128 rows each has
// rows of its own and takes every tile; otherwise they share the rows, and take
// every other tile each (the first half joins both parts in the end).
struct Halves {
  int n, T;
  bool apart;             // rows of their own
  __device__ __forceinline__ Halves(int rows, int T_)
      : n(rows > kHalf || T_ > 1 ? 2 : 1), T(T_), apart(rows > kHalf) {}
  __device__ __forceinline__ int tiles(int h) const {
    return apart ? T : (T + 1 - h) / 2;
  }
  // tile i of half h among the segment's
  __device__ __forceinline__ int tile(int h, int i) const {
    return apart ? i : 2 * i + h;
  }
};

// A row of the segment as its thread sees it.
struct Row {
  int out;        // row of out and lse, -1: none
  int lim;        // tokens it sees
};
__device__ __forceinline__ Row row_at(const PagedAttnArgs& a, const Shape& s,
                                      const Segment& g, int r) {
  if (r >= g.rows) return Row{-1, 0};
  const int query = (g.row0 + r) / s.g;       // of all sequences
  const int b = query / a.Q, i = query - b * a.Q;
  bool bad = false;
  const Lens l = lens_of(a, b, &bad);
  if (i >= l.nq) return Row{-1, 0};
  const int lim = a.causal ? min(l.n, l.n - l.nq + i + 1) : l.n;
  return Row{query * a.Hq + g.hk * s.g + (g.row0 + r) - query * s.g,
             min(lim, g.end)};
}

__global__ void __launch_bounds__(kThreads, 1)
    shared_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v,
                          const __grid_constant__ PagedAttnArgs a,
                          const Shape shape, void* ws) {
  // (all there is: no room to align it by hand)
  extern __shared__ __align__(1024) uint8_t base[];
  uint8_t* sq = base;                         // [2 halves][2][128][128]
  uint8_t* wide = sq + kQBytes;               // [kWide][2][128][128]
  uint8_t* raw = wide + kWide * kWideBytes;   // [kRaw][128][128]
  Meta& m = *reinterpret_cast<Meta*>(raw + kRaw * kRawBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &m.abort;

  if (tid == 0) {
    for (int i = 0; i < kRaw; ++i) {
      tc::mbar_init(&m.raw_full[i], 1);
      tc::mbar_init(&m.raw_empty[i], 4);
    }
    for (int i = 0; i < kWide; ++i) {
      tc::mbar_init(&m.wide_full[i], 4);
      tc::mbar_init(&m.wide_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&m.s_full[i], 2);
      tc::mbar_init(&m.p_full[i], 4);
      tc::mbar_init(&m.q_full[i], 4);
      tc::mbar_init(&m.o_full[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(&m.seg_full[i], 1);
      tc::mbar_init(&m.seg_empty[i], 1 + 1 + 4 + 8);
    }
    tc::mbar_init(&m.x_full, 4);
    tc::mbar_init(&m.x_empty, 4);
    tc::mbar_init(&m.drain, 1);
    m.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&m.tmem, 512);
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
  const int steps = a.D / 16;                 // 16 dimensions
  pdl_wait();
  pdl_trigger();

  Ring<kSegs> rg;
  // the next segment; false: something gave up
  auto next_segment = [&] {
    const bool ok = wait_for(&m.seg_full[rg.at], rg.phase, abort, a.wait_ns);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  auto done_segment = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&m.seg_empty[rg.at]);
    rg.next();
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int pt = kTile / a.page;            // pages of a tile
    const int oob = a.num_pages * a.Hkv * a.page;  // a row past the pool
    const uint32_t box = (uint32_t)a.page * 128;
    const float c = fabsf(a.scale) * kLog2e;
    Ring<kRaw> rr;
    int in_flight = 0, tile = 0;
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const Segment g = m.seg[rg.at];
      done_segment();
      if (g.done) break;
      const int pages = (g.end + a.page - 1) / a.page;
      const int last = min(pages, g.tok0 / a.page + g.T * pt);
      // page ids two chunks of 32 ahead, their scales one ahead
      int at = g.tok0 / a.page;
      auto load_id = [&](int first) {
        const int pg = first + lane;
        return pg < last ? a.table[(size_t)g.b * a.max_pages + pg] : -1;
      };
      auto load_scale = [&](const float* s, int pid) {
        return pid >= 0 && pid < a.num_pages
                   ? s[(size_t)pid * a.Hkv + g.hk] : 1.f;
      };
      int id = load_id(at), id1 = load_id(at + 32), id2 = load_id(at + 64);
      float ks = load_scale(a.k_scale, id), vs = load_scale(a.v_scale, id);
      float ks1 = load_scale(a.k_scale, id1), vs1 = load_scale(a.v_scale, id1);
      float top_lv = -INFINITY;               // of the pages so far
      for (int t = 0; t < g.T && ok; ++t) {
        const int pg = g.tok0 / a.page + t * pt;  // first page of the tile
        if (pg - at == 32) {
          at += 32;
          id = id1; ks = ks1; vs = vs1;
          id1 = id2;
          ks1 = load_scale(a.k_scale, id1);
          vs1 = load_scale(a.v_scale, id1);
          id2 = load_id(at + 64);
        }
        const int from = pg - at + lane;      // lane < pt: its page
        const int pid = __shfl_sync(0xffffffffu, id, from & 31);
        const float pk = __shfl_sync(0xffffffffu, ks, from & 31);
        const float pv = __shfl_sync(0xffffffffu, vs, from & 31);
        const bool have = lane < pt && pg + lane < last;
        const bool bad = have && (pid < 0 || pid >= a.num_pages);
        if (bad) raise_error(a.err, kErrBadIndex);
        const int row = bad ? oob : (pid * a.Hkv + g.hk) * a.page;
        const uint32_t bytes = box * __popc(__ballot_sync(0xffffffffu, have));
        const float lv = fminf(fmaxf(log2f(pv), kLeastLv), kMostLv);
        top_lv = fmaxf(top_lv, warp_top(have ? lv : -INFINITY));
        // every 16 tokens have their page's (lanes 0 to 7)
        {
          const int page_of = lane * 16 / a.page;  // (below pt, lane < 8)
          const float k16 = __shfl_sync(
              0xffffffffu, have && !bad ? pk * c : 0.f, page_of & 31);
          const float l16 =
              __shfl_sync(0xffffffffu, have ? lv : 0.f, page_of & 31);
          if (lane < kTile / 16)
            m.info[tile % kInfo][lane] = make_float4(
                k16, l16,
                l16 < top_lv - kFarLv ? 0.f : tc::ex2_approx(kSumRef - l16),
                0.f);
        }
        ++tile;
        __syncwarp();
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && wait_for(&m.raw_empty[rr.at], rr.phase ^ 1, abort,
                              a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(&m.raw_full[rr.at], bytes);
          __syncwarp();
          if (have)
            tc::tma_load_2d(raw + rr.at * kRawBytes + lane * box,
                            kv ? &map_v : &map_k, &m.raw_full[rr.at], 0, row);
          rr.next();
          in_flight = min(in_flight + 1, kRaw);
        }
      }
    }
    // no copy is in flight when the CTA leaves, whatever the others did
    int never = 0;
    for (; in_flight > 0; --in_flight) {
      Ring<kRaw> r = rr;
      r.at -= in_flight;
      if (r.at < 0) {
        r.at += kRaw;
        r.phase ^= 1;
      }
      wait_for(&m.raw_full[r.at], r.phase, &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp waits, one elected thread issues: operands stay in uniform
    // registers.  Products are issued as what they wait for is there, either
    // half's: scores go to the columns that weights leave, and products of
    // different shapes are not ordered, so those with the weights have to be
    // done before.
    const uint32_t tm = uniform(tmem);
    constexpr uint32_t id_s = idesc_f16(kTile);
    const uint32_t id_o = idesc_f16_mn(a.D);
    bool ok = true;
    uint32_t wide_at = 0;                     // operands before the segment's
    uint32_t n0 = 0, n1 = 0;                  // the halves' tiles before it
    uint32_t q_par0 = 0, q_par1 = 0;
    while (ok) {
      if (!next_segment()) break;
      const bool done = m.seg[rg.at].done;
      const int T = uniform(m.seg[rg.at].T);
      const Halves hv(uniform(m.seg[rg.at].rows), T);
      done_segment();
      if (done) break;
      auto ready = [&](uint64_t* bar, uint32_t par) {
        return __all_sync(0xffffffffu, test_wait(bar, par)) != 0;
      };
      // A stage is free when both halves have used it, or the one that does.
      auto release = [&](uint32_t at) {
        tc::mma_commit(&m.wide_empty[at]);
        if (!hv.apart) tc::mbar_arrive(&m.wide_empty[at]);
      };
      // Scores (`next` even) and values (odd) of a half's tiles by turns, the
      // halves by turns; one piece of code for both.
      int h = 0, next = 0, next_o = 0;        // this half's, the other's
      uint32_t n = n0, n_o = n1, q_par = q_par0, q_par_o = q_par1;
      uint32_t full_to = wide_at;             // operands known to be there
      uint64_t since = 0;                     // when something was issued last
      int polls = 0;
      while (next < 2 * hv.tiles(h) || next_o < 2 * hv.tiles(1 - h)) {
        const int i = next >> 1;
        bool go = i < hv.tiles(h);
        if (go) {
          const int t = hv.tile(h, i);
          const uint32_t seq = wide_at + 2 * t + (next & 1), at = seq % kWide;
          if (next & 1)
            go = ready(&m.p_full[h], (n + i) & 1);
          else
            go = i == 0 ? ready(&m.q_full[h], q_par)
                        : ready(&m.o_full[h], (n + i - 1) & 1);
          if (go && seq >= full_to) {         // (they come in order)
            go = ready(&m.wide_full[at], (seq / kWide) & 1);
            if (go) full_to = seq + 1;
          }
          if (go) {
            tc::fence_after_sync();
            const uint32_t src = uniform(tc::smem_u32(wide) + at * kWideBytes);
            const uint32_t ds = uniform(tm + h * kTile);
            if (next & 1) {
              const uint64_t dv = sdesc_mn_wide(src);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                  mma_f16_ts(ds + kRows, ds + 8 * k, dv + k * (2048 >> 4),
                             id_o, i > 0 || k > 0);
                release(at);
                tc::mma_commit(&m.o_full[h]);
              }
            } else {
              if (i == 0) q_par ^= 1;
              const uint64_t dk = tc::sdesc_k_sw128(src);
              const uint64_t dq = tc::sdesc_k_sw128(
                  uniform(tc::smem_u32(sq) + h * (kQBytes / 2)));
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const int off = (k >> 2) * (kRawBytes >> 4) + (k & 3) * 2;
                  if (k < steps)
                    tc::mma_bf16(ds, dq + off, dk + off, id_s, k > 0);
                }
                release(at);
                tc::mma_commit(&m.s_full[h]);
                tc::mbar_arrive(&m.s_full[h]);  // (releases the tile's scales)
              }
            }
            __syncwarp();
            ++next;
            polls = 0;
            since = 0;
          }
        }
        if (!go && ++polls >= (a.wait_ns < 1000000ull ? 2 : 256)) {
          polls = 0;
          const uint64_t now = tc::globaltimer_ns();
          if (since == 0) since = now;
          if (*abort || now - since > a.wait_ns) {
            *abort = 1;
            ok = false;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        h ^= 1;
        const int k = next;
        next = next_o;
        next_o = k;
        const uint32_t k1 = n, k2 = q_par;
        n = n_o;
        n_o = k1;
        q_par = q_par_o;
        q_par_o = k2;
      }
      q_par0 = h ? q_par_o : q_par;
      q_par1 = h ? q_par : q_par_o;
      wide_at += 2 * T;
      n0 += hv.tiles(0);
      n1 += hv.tiles(1);
    }
    if (elect_one()) tc::mma_commit(&m.drain);
    __syncwarp();
    int never = 0;
    wait_for(&m.drain, 0, &never, kWaitLimitNs);
  } else if (warp == 2) {
    // ----------------------------------------------------------- the run
    Walk w;
    const Parts parts = parts_of(ws, (size_t)a.B * a.Q * a.Hq, a.D);
    {
      bool bad = false;
      walk_start(a, shape, blockIdx.x, gridDim.x, w, &bad);
      if (blockIdx.x == 0) {
        if (bad) raise_error(a.err, kErrBadIndex);
        if (lane == 0) *parts.runs = w.runs;
      }
    }
    // (to the end even if something gave up: the join reads what units left)
    bool ok = true;
    for (bool more = true; more;) {
      ok = ok && wait_for(&m.seg_empty[rg.at], rg.phase ^ 1, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      Segment g;
      more = walk_next(a, shape, w, blockIdx.x, g, parts.begun);
      if (!ok) continue;
      if (lane == 0) {
        m.seg[rg.at] = g;
        tc::mbar_arrive(&m.seg_full[rg.at]);
      }
      __syncwarp();
      rg.next();
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------- converters
    const int tok = tid - 128;                // row of the tile
    Ring<kRaw> rr;
    Ring<kWide> rw;
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const int done = m.seg[rg.at].done, T = m.seg[rg.at].T;
      int left = m.seg[rg.at].end - m.seg[rg.at].tok0 - tok;
      done_segment();
      if (done) break;
      for (int t = 0; t < T && ok; ++t, left -= kTile) {
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          ok = ok && wait_for(&m.raw_full[rr.at], rr.phase, abort, a.wait_ns) &&
               wait_for(&m.wide_empty[rw.at], rw.phase ^ 1, abort, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint8_t* src = raw + rr.at * kRawBytes + tok * 128;
          uint8_t* dst = wide + rw.at * kWideBytes + tok * 128;
          // values past the cache's end may be anything: they are 0
          const bool live = left > 0;
          uint4 w[8];                         // (dimensions past D: zeros)
#pragma unroll
          for (int c = 0; c < 8; ++c)
            w[c] = *reinterpret_cast<const uint4*>(src +
                                                   ((c ^ (tok & 7)) << 4));
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (!live) w[c] = make_uint4(0, 0, 0, 0);
            const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                  (__nv_fp8x2_storage_t)(x[i >> 1] >> (16 * (i & 1))),
                  __NV_E4M3);
              y[i] = (uint32_t)h.x | (uint32_t)h.y << 16;
            }
            uint8_t* to = dst + (c >> 2) * kRawBytes;
            const int c0 = (c & 3) * 2;
            *reinterpret_cast<uint4*>(to + ((c0 ^ (tok & 7)) << 4)) =
                make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(to + (((c0 + 1) ^ (tok & 7)) << 4)) =
                make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_async();
          __syncwarp();
          if (lane == 0) {
            tc::mbar_arrive(&m.raw_empty[rr.at]);
            tc::mbar_arrive(&m.wide_full[rw.at]);
          }
          rr.next();
          rw.next();
        }
      }
    }
  } else if (warp >= 8) {
    // -------------------------------------------------------------- softmax
    const int half = (warp - 8) >> 2, quarter = warp & 3;
    const int r_half = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t s_col = lanes + half * kTile;
    const uint32_t o_col = lanes + kRows + half * kTile;
    uint8_t* qh = sq + half * (kQBytes / 2);
    const Parts parts = parts_of(ws, (size_t)a.B * a.Q * a.Hq, a.D);
    uint32_t n = 0;                           // tiles of this half
    uint32_t x_par = 0;
    bool lent = false;                        // the first half reads this O
    int tile = 0;                             // tiles before the segment's
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const Segment g = m.seg[rg.at];
      done_segment();
      if (g.done) break;
      const Halves hv(g.rows, g.T);
      const int tile0 = tile;
      tile += g.T;
      if (half >= hv.n) continue;
      const int r_unit = r_half + (hv.apart ? half * kHalf : 0);
      const Row row = row_at(a, shape, g, r_unit);
      float back = 0.f;                       // undoes the row's scaling
      // ---- q: eight lanes to a row, 16 dimensions each --------------------
      {
        const int ch = lane & 7;
#pragma unroll 1
        for (int j0 = 0; j0 < 8; j0 += 4) {
          uint4 u[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int from = (j0 + j) * 4 + (lane >> 3);
            const int out = __shfl_sync(0xffffffffu, row.out, from);
            u[j][0] = u[j][1] = make_uint4(0, 0, 0, 0);
            if (out >= 0 && ch < steps) {
              const uint4* src = reinterpret_cast<const uint4*>(
                  static_cast<const uint8_t*>(a.q) +
                  ((size_t)out * a.D + ch * 16) * 2);
              u[j][0] = __ldg(src);
              u[j][1] = __ldg(src + 1);
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v[8] = {u[j][0].x, u[j][0].y, u[j][0].z, u[j][0].w,
                                   u[j][1].x, u[j][1].y, u[j][1].z, u[j][1].w};
            float top = 0.f;                  // infinite: a NaN
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float x0 = __uint_as_float(v[k] << 16);
              const float x1 = __uint_as_float(v[k] & 0xffff0000u);
              top = x0 == x0 ? fmaxf(top, fabsf(x0)) : INFINITY;
              top = x1 == x1 ? fmaxf(top, fabsf(x1)) : INFINITY;
            }
#pragma unroll
            for (int o = 4; o; o >>= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e =
                max((int)(__float_as_uint(top) >> 23) - 127, -100);
            float up = top < INFINITY ? __uint_as_float((141 - e) << 23)
                                      : __uint_as_float(0x7fffffffu);
            if (a.scale < 0.f) up = -up;
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 h = __floats2half2_rn(
                  __uint_as_float(v[k] << 16) * up,
                  __uint_as_float(v[k] & 0xffff0000u) * up);
              y[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            const int r = quarter * 32 + (j0 + j) * 4 + (lane >> 3);
            if (ch < steps) {
              uint8_t* to = qh + (ch >> 2) * kRawBytes + r * 128;
              const int c0 = (ch & 3) * 2;
              *reinterpret_cast<uint4*>(to + ((c0 ^ (r & 7)) << 4)) =
                  make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(to + (((c0 + 1) ^ (r & 7)) << 4)) =
                  make_uint4(y[4], y[5], y[6], y[7]);
            }
            // the row's own thread keeps what undoes its scaling
            const float of = __shfl_sync(
                0xffffffffu, __uint_as_float((113 + e) << 23), (lane & 3) * 8);
            if ((lane >> 2) == j0 + j) back = of;
          }
        }
      }
      tc::fence_before_sync();                // (the last segment's O is read)
      fence_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&m.q_full[half]);
      const int lim = row.out >= 0 ? row.lim : 0x7fffffff;
      uint64_t l2 = 0;                        // two sums of weights
      float nr = 0.f;                         // -reference
      for (int i = 0; i < hv.tiles(half); ++i, ++n) {
        const int t = hv.tile(half, i);
        // (also says that the products before are done)
        ok = wait_for(&m.s_full[half], n & 1, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc::fence_after_sync();
        const float4* info = m.info[(tile0 + t) % kInfo];
        const int seen = lim - (g.tok0 + t * kTile);  // columns [0, seen)
        const bool masked = __any_sync(0xffffffffu, seen < kTile);
        // Half of the scores at a time, in loops that are not unrolled: two
        // warps of every scheduler run this code at different places, and
        // with all of it unrolled they waited for instructions.
        float y[kTile / 2];
        auto load = [&](int c0) {
#pragma unroll
          for (int c = 0; c < kTile / 2; c += 16)
            tmem_ld_x16(s_col + c0 + c,
                        *reinterpret_cast<float (*)[16]>(y + c));
          tmem_loaded(y);
        };
        // ---- the largest exponent ------------------------------------------
        float top = -INFINITY;
        bool far = false;
#pragma unroll 1
        for (int c0 = 0; c0 < kTile; c0 += kTile / 2) {
          load(c0);
          if (masked) {                       // for the second reading, too
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < kTile / 2; ++j) {
              if (c0 + j >= seen) y[j] = -INFINITY;
              w[j & 15] = __float_as_uint(y[j]);
              if ((j & 15) == 15) tmem_st_x16(s_col + c0 + j - 15, w);
            }
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float4 k = info[c0 / 16 + b];
            const float* z = y + 16 * b;
            float big[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              big[j] = fmaxf(fmaxf(z[j], z[4 + j]), fmaxf(z[8 + j], z[12 + j]));
            big[0] = fmaxf(fmaxf(big[0], big[1]), fmaxf(big[2], big[3]));
            top = fmaxf(top, fmaf(big[0], factor(k.x * back), k.y));
            far |= k.z == 0.f;
          }
        }
        if (masked) tmem_stored();
        if (__any_sync(0xffffffffu, i == 0 || top + nr > kRaise)) {
          // ---- raise the reference: nothing to raise for a row that sees
          // nothing, and in the first tile nothing to scale
          float d = 0.f;
          if (top > -INFINITY && (i == 0 || top + nr > kHead))
            d = kHead - ceilf(top + nr);
          nr += d;
          if (i > 0) {
            // in two factors: the sum may hold what the weights do not
            const float f = tc::ex2_approx(fmaxf(d, -100.f));
            const float f2 = tc::ex2_approx(fminf(d + 100.f, 0.f));
            l2 = mul2(mul2(l2, pack2(f, f)), pack2(f2, f2));
#pragma unroll 1
            for (int c = 0; c < steps; ++c) {
              float o[16];
              tmem_ld_x16(o_col + 16 * c, o);
              tmem_loaded(o);
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[j] = __float_as_uint(o[j] * f * f2);
              tmem_st_x16(o_col + 16 * c, w);
            }
          }
        }
        if (far) {                            // (the same in all threads)
#pragma unroll 1
          for (int c = 0; c < kTile; c += 16) {
            const float4 k = info[c / 16];
            if (k.z != 0.f) continue;
            float z[16];
            tmem_ld_x16(s_col + c, z);
            tmem_loaded(z);
            const float f = factor(k.x * back), apart = nr + kSumRef;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              sum += tc::ex2_approx(fmaf(z[j], f, apart));
            l2 = add2(l2, pack2(sum, 0.f));
          }
        }
        // ---- the weights ---------------------------------------------------
#pragma unroll 1
        for (int c0 = 0; c0 < kTile; c0 += kTile / 2) {
          load(c0);
#pragma unroll
          for (int c = 0; c < kTile / 2; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float4 k = info[(c0 + c) / 16 + b];
              const float* z = y + c + 16 * b;
              const float f = factor(k.x * back), add = k.y + nr;
              const uint64_t f2 = pack2(f, f), a2 = pack2(add, add);
              uint64_t sum[2];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                float e0, e1;
                unpack2(fma2(pack2(z[2 * j], z[2 * j + 1]), f2, a2), e0, e1);
                e0 = tc::ex2_approx(e0);
                e1 = tc::ex2_approx(e1);
                const uint64_t e = pack2(e0, e1);
                sum[j & 1] = j < 2 ? e : add2(sum[j & 1], e);
                const __half2 h = __floats2half2_rn(e0, e1);
                w[8 * b + j] = *reinterpret_cast<const uint32_t*>(&h);
              }
              l2 = fma2(add2(sum[0], sum[1]), pack2(k.z, k.z), l2);
            }
            // (onto scores that have been read)
            tmem_st_x16(s_col + (c0 + c) / 2, w);
          }
        }
        tmem_stored();
        if (lent) {                           // O may be written again?
          lent = false;
          ok = wait_for(&m.x_empty, x_par, abort, a.wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          x_par ^= 1;
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.p_full[half]);
      }
      if (!ok) break;
      // ---- the part ----------------------------------------------------------
      ok = wait_for(&m.o_full[half], (n - 1) & 1, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      float l, l_odd;
      unpack2(l2, l, l_odd);
      l += l_odd;
      // The halves' parts of the same rows lie in the same lanes: the first half
      // reads both, against the larger of the references.
      const bool both = hv.n == 2 && !hv.apart;
      float d0 = 0.f, d1 = 0.f;               // to it
      if (both && half == 1) {
        m.x[r_half] = make_float2(l, nr);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.x_full);
        lent = true;
        continue;
      }
      if (both) {
        ok = wait_for(&m.x_full, x_par, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        x_par ^= 1;
        tc::fence_after_sync();
        const float2 x = m.x[r_half];
        const bool on0 = l > 0.f || l != l, on1 = x.x > 0.f || x.x != x.x;
        const float to = on0 && on1 ? fminf(nr, x.y) : on0 ? nr : x.y;
        d0 = on0 ? to - nr : -INFINITY;
        d1 = on1 ? to - x.y : -INFINITY;
        auto scaled = [](float v, float d) {
          return d == -INFINITY ? 0.f
                                : v * tc::ex2_approx(fmaxf(d, -100.f)) *
                                      tc::ex2_approx(fminf(d + 100.f, 0.f));
        };
        l = scaled(l, d0) + scaled(x.x, d1);
        nr = to;
      }
      const bool any = l > 0.f || l != l;     // a NaN stays one
      // l = frac 2^ex; 2^ref: what frac counts
      const int ex = min(max((int)(__float_as_uint(l) >> 23) - 127, -100), 120);
      const float f0 = tc::ex2_approx(d0 + (kSumRef - (float)ex));
      const float f1 = tc::ex2_approx(d1 + (kSumRef - (float)ex));
      const size_t rows = (size_t)a.B * a.Q * a.Hq;
      const size_t at =
          g.slot >= 0 ? (size_t)g.slot * kRows + r_unit
                      : parts.by_row + (g.prefix ? 0 : rows) + row.out;
      if (row.out >= 0)
        parts.ml[at] = make_float2(
            any ? (float)ex - nr - kSumRef : -INFINITY,
            any ? l * __uint_as_float((127 - ex) << 23) : 0.f);
#pragma unroll 1
      for (int c = 0; c < steps; ++c) {
        float o[16], o1[16];
        tmem_ld_x16(o_col + 16 * c, o);
        if (both) {
          tmem_ld_x16(o_col + kTile + 16 * c, o1);
          tmem_loaded(o1);
        }
        tmem_loaded(o);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          o[j] *= f0;
          if (both) o[j] = fmaf(o1[j], f1, o[j]);
        }
        if (row.out >= 0) {
          float4* to = reinterpret_cast<float4*>(parts.o + at * a.D + 16 * c);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            to[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2],
                                o[4 * j + 3]);
        }
        __syncwarp();
      }
      if (both) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.x_empty);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
  if (tid == 0 && m.abort) raise_error(a.err, kErrTimeout);
}

// Joins the parts of every row of out: a warp each.
constexpr int kJoinWarps = 4;
constexpr int kMostParts = 2 * kMaxCtas;
__global__ void __launch_bounds__(32 * kJoinWarps)
    shared_attn_tc_join_kernel(const __grid_constant__ PagedAttnArgs a,
                               const Shape s, void* ws) {
  __shared__ int s_at[kJoinWarps][kMostParts];
  __shared__ float s_w[kJoinWarps][kMostParts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  const int rows = a.B * a.Q * a.Hq;
  const int row = blockIdx.x * kJoinWarps + warp;
  if (row >= rows) return;
  const Parts parts = parts_of(ws, rows, a.D);
  const int query = row / a.Hq, h = row - query * a.Hq;
  const int b = query / a.Q, i = query - b * a.Q, hk = h / s.g;
  bool bad = false;
  const Lens l = lens_of(a, b, &bad);
  const Runs runs = *parts.runs;
  int n = 0;
  // the parts of row r of a unit; whole: where the row's part of all of it is
  auto add = [&](int at_b, int u, int cost, int r, size_t whole) {
    const Begun g = parts.begun[unit_of(s, a.Hkv, at_b, hk, u)];
    const int work = work_of(g.T, cost);
    // (in range whatever another call has left in a workspace that is its own
    // at the same time)
    const int c1 = min(g.c1, kMaxCtas - 1);
    for (int c = max(g.c0, 0) + lane; c - lane <= c1; c += 32) {
      int at = -1;
      if (c <= c1) {
        const int p0 = max(0, runs.start(c) - g.first);
        const int p1 = min(work, runs.start(c + 1) - g.first);
        const int t0 = tiles_before(p0, g.T, cost);
        const int t1 = tiles_before(p1, g.T, cost);
        if (t1 > t0)
          at = t1 - t0 == g.T ? (int)whole
                              : (2 * c + (p0 > 0 ? 0 : 1)) * kRows + r;
      }
      const uint32_t have = __ballot_sync(0xffffffffu, at >= 0);
      if (at >= 0) s_at[warp][n + __popc(have & ((1u << lane) - 1))] = at;
      n += __popc(have);
    }
  };
  if (i < l.nq) {
    const int r_own = i * s.g + h - hk * s.g, r_all = b * s.own + r_own;
    const int u = r_all / kRows, v = r_own / kRows;
    if (s.tiles > 0)
      add(-1, u, cost_of(s.all, u), r_all % kRows, parts.by_row + row);
    if (s.own_units == 0) {                   // another launch's, by row
      if (lane == 0) s_at[warp][n] = (int)(parts.by_row + rows + row);
      ++n;
    } else if (tiles_of(a, s, l, v) > 0) {
      add(b, v, cost_of(s.own, v), r_own % kRows, parts.by_row + rows + row);
    }
  }
  __syncwarp();
  float top = -INFINITY;
  for (int k = lane; k < n; k += 32)
    top = fmaxf(top, parts.ml[s_at[warp][k]].x);
  top = warp_max(top);
  float sum = 0.f;
  for (int k = lane; k < n; k += 32) {
    const float2 v = parts.ml[s_at[warp][k]];
    const float w = v.x == -INFINITY ? 0.f : exp2f(v.x - top);
    s_w[warp][k] = w;
    sum += w * v.y;
  }
  sum = warp_sum(sum);
  __syncwarp();
  const bool on = sum > 0.f || sum != sum;
  const float inv = on ? 1.f / sum : 0.f;
  if (lane == 0 && a.lse)
    a.lse[row] = on ? (log2f(sum) + top) * 0.6931471805599453f : -INFINITY;
  if (4 * lane >= a.D) return;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAt = 8;                      // parts on their way at once
  for (int k0 = 0; k0 < n; k0 += kAt) {
    float4 v[kAt];
    float w[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      w[j] = k0 + j < n ? s_w[warp][k0 + j] : 0.f;
      v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (w[j] != 0.f)                        // (a NaN is none)
        v[j] = *reinterpret_cast<const float4*>(
            parts.o + (size_t)s_at[warp][k0 + j] * a.D + 4 * lane);
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      o.x = fmaf(w[j], v[j].x, o.x);
      o.y = fmaf(w[j], v[j].y, o.y);
      o.z = fmaf(w[j], v[j].z, o.z);
      o.w = fmaf(w[j], v[j].w, o.w);
    }
  }
  const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 v;
  v.x = *reinterpret_cast<const uint32_t*>(&x);
  v.y = *reinterpret_cast<const uint32_t*>(&y);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                            (size_t)row * a.D + 4 * lane) = v;
}

Shape shape_of(const PagedAttnArgs& a, int shared) {
  Shape s;
  s.g = a.Hq / a.Hkv;
  s.own = a.Q * s.g;
  s.all = a.B * s.own;
  s.own_units = (s.own + kRows - 1) / kRows;
  s.all_units = (s.all + kRows - 1) / kRows;
  s.shared = shared;
  s.tiles = (shared + kTile - 1) / kTile;
  return s;
}

// What the parts and tables take.
size_t tc_ws(long long B, long long Q, int Hq, int Hkv, int D) {
  const size_t n = (size_t)2 * kMaxCtas * kRows + 2 * (size_t)(B * Q * Hq);
  const long long own = Q * (Hq / Hkv);
  const size_t units = Hkv * ((B * own + kRows - 1) / kRows +
                              B * ((own + kRows - 1) / kRows));
  const size_t need =
      n * (D * sizeof(float) + sizeof(float2)) + 32 + units * sizeof(Begun);
  return (need + 255) & ~(size_t)255;
}

}  // namespace

size_t shared_attn_tc_ws(long long B, long long Q, int Hq, int Hkv, int D) {
  return tc_ws(B, Q, Hq, Hkv, D) + paged_attn_tc_ws((int)B, (int)Q, Hq, Hkv);
}

cudaError_t launch_shared_attn_tc(const PagedAttnArgs& a, int shared, int sms,
                                  void* ws, cudaStream_t stream) {
  // Few tiles of shared tokens are read for each sequence again by the kernel
  // whose cost follows the rows.  Each costs it 0.7 us with 16 rows and 1.1 with
  // 48, and a call 8 us less: up to 28 tiles of 16 rows a CTA.  (32 query and 8
  // key heads: 4 sequences, 2148 tokens 14.7 against 22.9 us; 2 and 4 sequences,
  // 16884 tokens, 13 and 27 tiles a CTA 21.7 and 31.0 against 32.4 and 35.1, 8
  // sequences 51.1 against 38.1; 16 sequences with 9 queries, 2148 tokens, 13
  // tiles of 48 rows 35.8 against 36.9.)
  Shape s = shape_of(a, shared);
  const PagedTcUnits units = paged_attn_tc_units(a.Q, a.Hq, a.Hkv);
  const long long n_units = (long long)a.B * a.Hkv * units.row_tiles;
  if (n_units * s.tiles * units.N <= 448ll * sms)
    return launch_paged_attn_tc(a, sms, static_cast<float*>(ws), stream,
                                shared);
  const long long own_tiles =
      ((long long)a.max_pages * a.page - shared + kTile - 1) / kTile;
  const long long most =
      a.Hkv * (long long)s.all_units * (kUnitCost + 2ll * s.tiles) +
      (long long)a.B * a.Hkv * s.own_units * (kUnitCost + 2 * own_tiles);
  const long long rows = (long long)a.B * a.Q * a.Hq;
  // (and the parts' numbers stay within 32 bits)
  if (most > 0x7fffffffll || 2 * rows + 2 * kMaxCtas * kRows > 0x7fffffffll)
    return cudaErrorNotSupported;
  // Own tokens of few rows fill a tile of 128 rows badly: where there are many
  // such units that kernel takes them, in a launch (and a join) more.  (64
  // sequences, 32 query heads: 16384 shared and 500 to 1000 own tokens 96.6
  // against 99.2 us, 64 heads and 1000 to 2000 own ones 129 against 150; 256
  // sequences, 1024 and 50 to 100 tokens 91 against 147.  16 sequences, 16384
  // and 250 to 500 tokens: 50.0 against 42.8.)
  const bool apart =
      units.N <= kPagedTcOwnRows && n_units >= 2 * sms;
  if (apart) s.own_units = 0;
  const int G = std::min(sms, kMaxCtas);
  CUtensorMap mk, mv;
  const uint64_t pool = (uint64_t)a.num_pages * a.Hkv * a.page;
  if (!make_tmap_u8_2d(&mk, a.k_codes, a.D, pool, 128, a.page) ||
      !make_tmap_u8_2d(&mv, a.v_codes, a.D, pool, 128, a.page))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(
      shared_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      kSmem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(G), dim3(kThreads), kSmem, stream);
  e = cudaLaunchKernelEx(&L.cfg, shared_attn_tc_kernel, mk, mv, a, s, ws);
  if (e != cudaSuccess) return e;
  if (apart) {
    const Parts parts = parts_of(ws, rows, a.D);
    PagedAttnArgs own = a;
    own.out = parts.o + (parts.by_row + rows) * a.D;
    own.lse = reinterpret_cast<float*>(parts.ml + parts.by_row + rows);
    e = launch_paged_attn_tc(
        own, sms,
        reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                 tc_ws(a.B, a.Q, a.Hq, a.Hkv, a.D)),
        stream, shared, true);
    if (e != cudaSuccess) return e;
  }
  PdlLaunch J(dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)),
              dim3(32 * kJoinWarps), 0, stream);
  return cudaLaunchKernelEx(&J.cfg, shared_attn_tc_join_kernel, a, s, ws);
}

}  // namespace dflash
