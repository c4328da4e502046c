// The attention weight that cached tokens gather, on the tensor cores
// (tcgen05), for bf16 queries and heads of up to 128 dimensions.
//
// The cached codes go from HBM to the MMAs as they are, with q as the sum of two
// E4M3 numbers side by side in the MMA's N (a row's largest value scaled to
// [128, 256); the second part holds 2^5 times what the first leaves, in steps of
// 2^-14: all of bf16's bits of values from 2^-7 on, 2^-14 of the largest, and
// smaller ones to 2^-15, 2^-22 of it).  S^T[token, row] = K q^T, so a thread
// owns a token: its key's scale is one factor, and the sum over the rows is its
// own.  A row brings its scaling and its logsumexp (in bits).
//
// All tiles of 128 tokens of all (sequence, key head) pairs are numbered, and
// every CTA (one per SM) takes an equal run, counted with the rows that they
// have. With more than 128 rows the run's tiles are gone through for each 128
// rows again (the codes then come from L2) and the tokens' sums kept in shared
// memory meanwhile: one thread owns a token throughout, nothing is added
// atomically.
//
// Warps: 0 copies tiles (TMA, one box per page), 1 issues the MMAs, 2 hands out
// the segments, 4-7 lay out q (two buffers), the others take the tiles' weights:
// groups of four a tile each by turns, four groups with up to 64 rows (whose
// scores are 128 columns), else two.  What bounds it: the latencies of a tile's
// way through TMEM and these warps; HBM at 54 %.  32 sequences of up to 8000
// tokens with 36 rows 48 us (4.4 TB/s), 72 rows 73 us; one row of 20000 tokens
// 10.7 us, the chain of one tile; a prompt of 2048 tokens, four heads to a key
// head, 320 us (its rows are laid out 128 at a time, for one tile a CTA). (Two
// groups for 36 rows: 59 us.)
// Every wait is bounded; on a timeout the CTA stops issuing, drains, frees TMEM
// and flags the error word.
#include <cuda_fp8.h>

#include <algorithm>

#include "attn_roles.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace dflash {
namespace {

constexpr int kTile = 128;       // tokens of a tile
constexpr int kTileBytes = kTile * 128;
constexpr int kMaxRows = 128;    // of a segment
constexpr int kSegs = 4;
constexpr int kUnitCost = 2;     // of a pair besides its tiles, in tiles
constexpr float kLog2e = 1.4426950408889634f;
// A score is (sum of products) (key's factor) (row's factor), and the first two
// alone can pass fp32's range: 2^24 times a key's scale of up to 2^120.  So
// 2^24 goes from the key's factor to the row's, for queries below 2^111 (scores
// of larger ones pass 2^47 with the smallest scale, where fp32 has no weights).
constexpr int kToRow = 24;

// Tiles of one pair with (up to 64 or 128) of its rows; without rows: the sums
// of those tiles are complete.
struct Segment {
  int done;
  int b, hk;
  int row0, rows;
  int tok0, T, end;              // first token, tiles, end of the tokens
  int lone;                      // all rows: sums are complete at once
  int n, nq;
};
// Two rows: what undoes their scaling, and -logsumexp in bits.
struct alignas(16) Rows {
  float rel[2], nl[2];
};
// For segments of up to 64 rows, whose scores leave TMEM room for four tiles,
// or of up to 128.
template <int kRows_>
struct Plan {
  static constexpr int kRows = kRows_;
  static constexpr int kGroups = kRows == 64 ? 4 : 2;  // that take weights
  static constexpr int kThreads = 256 + 128 * kGroups;
  static constexpr int kColumns = 512 / kGroups;
  static constexpr int kStages = kRows == 64 ? 11 : 8;  // tiles in shared memory
  // tiles whose sums are kept (a multiple of kGroups); 64 are all rows
  static constexpr int kKeep = kRows == 64 ? 8 : 48;
  static constexpr int kQBytes = 2 * kRows * 128;       // two parts

  struct Meta {
    Segment seg[kSegs];
    Rows row[2][kRows / 2];
    int lim[2][kRows];             // tokens a row sees (none without weights)
    int4 off[2];                   // some row has none: of the warps that say so
    float ks[kStages][8];          // factors of a tile's pages
    float keep[kKeep][kTile];
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t s_full[kGroups], s_empty[kGroups], q_full[2], q_empty[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t drain;
    uint32_t tmem;
    int abort;
  };
  static constexpr int kSmem = 2 * kQBytes + kStages * kTileBytes +
                               ((int)sizeof(Meta) + 15) / 16 * 16;
  static_assert(kSmem <= 232448, "");
};

struct Shape {
  int g, first;                  // heads of a key head; first tile's token
  int rows;                      // most of a segment
};
struct Lens {
  int n, nq;
};
__device__ __forceinline__ Lens lens_of(const AttnMassArgs& a, int b,
                                        bool* bad) {
  Lens l;
  l.n = mass_length(a, b, bad);
  l.nq = attn_clamp(a.q_len ? a.q_len[b] : a.Q, a.Q, bad);
  return l;
}
__device__ __forceinline__ int tiles_of(const Shape& s, const Lens& l) {
  return (max(0, l.n - s.first) + kTile - 1) / kTile;
}
// Of a tile: the times it is gone through.
__device__ __forceinline__ int cost_of(const Shape& s, const Lens& l) {
  return max(1, (l.nq * s.g + s.rows - 1) / s.rows);
}
__device__ __noinline__ int work_of(const AttnMassArgs& a, const Shape& s,
                                    const Lens& l) {
  const int T = tiles_of(s, l);
  return T > 0 ? kUnitCost + T * cost_of(s, l) : 0;
}

// Walks the pairs from a position in the numbering.  Position kUnitCost + t c
// of a pair whose tiles cost c is its tile t.
struct Walk {
  int b, hk, at;                 // at: position in the pair
  int left;                      // positions left in this CTA's run
};
__device__ __noinline__ void walk_start(const AttnMassArgs& a, const Shape& s,
                                        int cta, int grid, Walk& w,
                                        bool* bad) {
  const int lane = threadIdx.x & 31;
  const int per = (a.B + 31) / 32;
  const int b0 = min(a.B, lane * per), b1 = min(a.B, b0 + per);
  int work = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b)
    work += a.Hkv * work_of(a, s, lens_of(a, b, bad));
  int run = work;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  const int total = __shfl_sync(0xffffffffu, run, 31);
  const int p0 = (int)((long long)total * cta / grid);
  w = Walk{0, 0, 0, (int)((long long)total * (cta + 1) / grid) - p0};
  if (w.left <= 0) return;                 // the same in every lane
  const bool mine = p0 >= run - work && p0 < run;
  int o = p0 - (run - work);
  if (mine) {
    int h = 1;
#pragma unroll 1
    for (w.b = b0; w.b < b1; ++w.b) {
      h = work_of(a, s, lens_of(a, w.b, bad));
      if (o < a.Hkv * h) break;
      o -= a.Hkv * h;
    }
    w.hk = o / h;
    o -= w.hk * h;
  }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  w.b = __shfl_sync(0xffffffffu, w.b, from);
  w.hk = __shfl_sync(0xffffffffu, w.hk, from);
  w.at = __shfl_sync(0xffffffffu, o, from);
}
// The next pair's tiles [t0, t0 + T) of the run; false at its end.
__device__ __noinline__ bool walk_next(const AttnMassArgs& a, const Shape& s,
                                       Walk& w, Segment& g, int& t0) {
  bool bad = false;
  while (w.left > 0) {
    const Lens l = lens_of(a, w.b, &bad);
    const int T = tiles_of(s, l), c = cost_of(s, l);
    const int work = T > 0 ? kUnitCost + T * c : 0;
    const int end = min(work, w.at + w.left);
    auto before = [&](int at) {
      return at <= kUnitCost ? 0 : min(T, (at - kUnitCost + c - 1) / c);
    };
    t0 = before(w.at);
    g.T = before(end) - t0;
    g.b = w.b;
    g.hk = w.hk;
    g.n = g.end = l.n;
    g.nq = l.nq;
    w.left -= end - w.at;
    w.at = end;
    if (end == work) {
      w.at = 0;
      if (++w.hk == a.Hkv) {
        w.hk = 0;
        ++w.b;
      }
    }
    if (g.T > 0) return true;
  }
  return false;
}

// kind::f8f6f4, E4M3, fp32 D: N known at run time only.
__device__ __forceinline__ uint32_t idesc_n(int N) {
  return tc::idesc_e4m3_f32(kTile, 0) | ((uint32_t)(N >> 3) << 17);
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

template <int kRows>
__global__ void __launch_bounds__(Plan<kRows>::kThreads, 1)
    attn_mass_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ AttnMassArgs a,
                        const Shape shape) {
  using PL = Plan<kRows>;
  using Meta = typename PL::Meta;
  constexpr int kThreads = PL::kThreads, kStages = PL::kStages;
  constexpr int kGroups = PL::kGroups, kQBytes = PL::kQBytes;
  constexpr int kKeep = PL::kKeep;
  extern __shared__ __align__(1024) uint8_t base[];
  uint8_t* sq = base;                        // [2 buffers][2 parts][rows][128]
  uint8_t* sk = sq + 2 * kQBytes;            // [kStages][128][128]
  Meta& m = *reinterpret_cast<Meta*>(sk + kStages * kTileBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &m.abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&m.k_full[i], 1);
      tc::mbar_init(&m.k_empty[i], 1 + 4);
    }
    for (int i = 0; i < kGroups; ++i) {
      tc::mbar_init(&m.s_full[i], 2);
      tc::mbar_init(&m.s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&m.q_full[i], 4);
      tc::mbar_init(&m.q_empty[i], 1 + 4 * kGroups);
    }
    for (int i = 0; i < kSegs; ++i) {
      tc::mbar_init(&m.seg_full[i], 1);
      tc::mbar_init(&m.seg_empty[i], 1 + 1 + 4 + 4 * kGroups);
    }
    tc::mbar_init(&m.drain, 1);
    m.abort = 0;
    tc::fence_mbar_init();
  }
  for (int i = tid; i < kKeep * kTile; i += kThreads) (&m.keep[0][0])[i] = 0.f;
  if (warp == 1) {
    tc::tmem_alloc(&m.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) tc::tma_prefetch_map(&map_k);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = m.tmem;
  pdl_wait();
  pdl_trigger();

  Ring<kSegs> rg;
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
    const int pt = kTile / a.page;           // pages of a tile
    const int first_page = a.first / a.page;  // (of those below, none is read)
    const int oob = a.num_pages * a.Hkv * a.page;  // a row past the pool
    const uint32_t box = (uint32_t)a.page * 128;
    const float c = fabsf(a.scale) * kLog2e * (1.f / (1 << kToRow));
    Ring<kStages> rk;
    int in_flight = 0;
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const Segment g = m.seg[rg.at];
      done_segment();
      if (g.done) break;
      if (g.rows == 0) continue;
      const int page0 = g.tok0 / a.page;
      const int last = min((g.end + a.page - 1) / a.page, page0 + g.T * pt);
      // page ids two chunks of 32 ahead, their scales one ahead
      int at = page0;
      auto load_id = [&](int first) {
        const int pg = first + lane;
        return pg < last ? a.table[(size_t)g.b * a.max_pages + pg] : -1;
      };
      auto load_scale = [&](int pid) {
        return pid >= 0 && pid < a.num_pages
                   ? a.k_scale[(size_t)pid * a.Hkv + g.hk] : 0.f;
      };
      int id = load_id(at), id1 = load_id(at + 32), id2 = load_id(at + 64);
      float ks = load_scale(id), ks1 = load_scale(id1);
#pragma unroll 1
      for (int t = 0; t < g.T && ok; ++t) {
        const int pg = page0 + t * pt;       // first page of the tile
        if (pg - at == 32) {
          at += 32;
          id = id1;
          ks = ks1;
          id1 = id2;
          ks1 = load_scale(id1);
          id2 = load_id(at + 64);
        }
        const int from = pg - at + lane;     // lane < pt: its page
        const int pid = __shfl_sync(0xffffffffu, id, from & 31);
        const bool have =
            lane < pt && pg + lane < last && pg + lane >= first_page;
        const bool bad = have && (pid < 0 || pid >= a.num_pages);
        if (bad) raise_error(a.err, kErrBadIndex);
        const int row = bad ? oob : (pid * a.Hkv + g.hk) * a.page;
        const uint32_t bytes = box * __popc(__ballot_sync(0xffffffffu, have));
        ok = wait_for(&m.k_empty[rk.at], rk.phase ^ 1, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) expect_tx(&m.k_full[rk.at], bytes);
        __syncwarp();
        if (have)                            // (the factors follow)
          tc::tma_load_2d(sk + rk.at * kTileBytes + lane * box, &map_k,
                          &m.k_full[rk.at], 0, row);
        const float pk = __shfl_sync(0xffffffffu, ks, from & 31);
        if (lane < pt) m.ks[rk.at][lane] = have && !bad ? pk * c : 0.f;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.k_full[rk.at]);
        rk.next();
        in_flight = min(in_flight + 1, kStages);
      }
    }
    // no copy is in flight when the CTA leaves, whatever the others did
    int never = 0;
    for (; in_flight > 0; --in_flight) {
      Ring<kStages> r = rk;
      r.at -= in_flight;
      if (r.at < 0) {
        r.at += kStages;
        r.phase ^= 1;
      }
      wait_for(&m.k_full[r.at], r.phase, &never, kWaitLimitNs);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t tm = uniform(tmem);
    const uint32_t sk_u = uniform(tc::smem_u32(sk));
    const uint32_t sq_u = uniform(tc::smem_u32(sq));
    const int steps = (a.D + 31) / 32;       // of 32 dimensions
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t par) {
      ok = ok && wait_for(bar, par, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    Ring<kStages> rk;
    Ring<2> rq;
    uint32_t pars = 0;                       // of the score buffers
    while (ok) {
      if (!next_segment()) break;
      const bool done = m.seg[rg.at].done;
      const int T = uniform(m.seg[rg.at].T), rows = uniform(m.seg[rg.at].rows);
      done_segment();
      if (done) break;
      if (rows == 0) continue;
      const uint32_t idesc = uniform(idesc_n(2 * ((rows + 7) / 8 * 8)));
      const uint64_t dq =
          tc::sdesc_k_sw128(uniform(sq_u + rq.at * kQBytes));
      if (!wait(&m.q_full[rq.at], rq.phase)) break;
#pragma unroll 1
      for (int t = 0; t < T && ok; ++t) {
        const int buf = t & (kGroups - 1);
        // (a buffer's first use finds it empty)
        if (!wait(&m.s_empty[buf], (pars >> buf & 1) ^ 1)) break;
        pars ^= 1u << buf;
        if (!wait(&m.k_full[rk.at], rk.phase)) break;
        tc::fence_after_sync();
        const uint32_t d = uniform(tm + buf * PL::kColumns);
        const uint64_t dk =
            tc::sdesc_k_sw128(uniform(sk_u + rk.at * kTileBytes));
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < steps)
              tc::mma_e4m3(d, dk + 2 * k, dq + 2 * k, idesc, k > 0);
          tc::mma_commit(&m.k_empty[rk.at]);
          tc::mma_commit(&m.s_full[buf]);
          tc::mbar_arrive(&m.s_full[buf]);   // (releases the tile's factors)
          if (t == T - 1) tc::mma_commit(&m.q_empty[rq.at]);
        }
        __syncwarp();
        rk.next();
      }
      rq.next();
    }
    if (elect_one()) tc::mma_commit(&m.drain);
    __syncwarp();
    int never = 0;
    wait_for(&m.drain, 0, &never, kWaitLimitNs);
  } else if (warp == 2) {
    // ------------------------------------------------------------- the run
    Walk w;
    bool bad = false;
    walk_start(a, shape, blockIdx.x, gridDim.x, w, &bad);
    if (bad && blockIdx.x == 0) raise_error(a.err, kErrBadIndex);
    bool ok = true;
    auto put = [&](const Segment& g) {
      ok = ok && wait_for(&m.seg_empty[rg.at], rg.phase ^ 1, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (lane == 0) {
        m.seg[rg.at] = g;
        tc::mbar_arrive(&m.seg_full[rg.at]);
      }
      __syncwarp();
      rg.next();
    };
    Segment g;
    int t0;
    g.done = 0;
#pragma unroll 1
    while (ok && walk_next(a, shape, w, g, t0)) {
      const int rows = g.nq * shape.g, all = g.T;
      g.lone = rows > 0 && rows <= kRows;
#pragma unroll 1
      for (int from = 0; from < all && ok; from += g.lone ? all : kKeep) {
        const int T = g.lone ? all : min(kKeep, all - from);
        g.tok0 = shape.first + (t0 + from) * kTile;
#pragma unroll 1
        for (int r = 0; r < rows && ok; r += kRows) {
          g.row0 = r;
          g.rows = min(kRows, rows - r);
          // tiles that the last of these rows sees
          const int i = (r + g.rows - 1) / shape.g;
          const int lim = a.causal ? g.n - g.nq + i + 1 : g.n;
          g.T = min(T, (max(0, lim - g.tok0) + kTile - 1) / kTile);
          if (g.T > 0) put(g);
        }
        if (!g.lone) {
          g.rows = 0;
          g.T = T;
          put(g);
        }
      }
    }
    g.done = 1;
    put(g);
  } else if (warp >= 4 && warp < 8) {
    // -------------------------------------------------------------- q's parts
    const int ch = tid & 7, r16 = (tid - 128) >> 3;  // 16 dimensions of a row
    Ring<2> rq;
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const Segment g = m.seg[rg.at];
      done_segment();
      if (g.done) break;
      if (g.rows == 0) continue;
      ok = wait_for(&m.q_empty[rq.at], rq.phase ^ 1, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      uint8_t* q = sq + rq.at * kQBytes;
      const int np = (g.rows + 7) / 8 * 8;   // rows of a part
      // All values fly at once, asynchronously, to where their codes will be:
      // the first 64 dimensions of a row in its first part, the others in its
      // second.  The lanes of a row read them before one writes.
      auto raw = [&](int r) {
        return q + (ch >> 2) * np * 128 + r * 128 + (ch & 3) * 32;
      };
      auto out_of = [&](int r) {
        const int row = g.row0 + r, i = row / shape.g;
        return (long long)((size_t)g.b * a.Q + i) * a.Hq + g.hk * shape.g +
               row - i * shape.g;
      };
      // A row whose logsumexp is infinite has no weights, whatever it holds: its
      // scores, which may be no numbers, are masked.
      bool off = false;
#pragma unroll 1
      for (int r = r16; r < np; r += 16) {
        const bool read = r < g.rows && ch * 16 < a.D;
        const long long out = out_of(r);
        const uint8_t* src = static_cast<const uint8_t*>(a.q) +
                             (read ? (out * a.D + ch * 16) * 2 : 0);
        copy16(tc::smem_u32(raw(r)), src, read);
        copy16(tc::smem_u32(raw(r) + 16), src + 16, read);
        if (ch == 0) {
          const float lse = r < g.rows ? a.lse[out] : -INFINITY;
          const bool none = fabsf(lse) == INFINITY;
          m.row[rq.at][r >> 1].nl[r & 1] = none ? -INFINITY : -lse * kLog2e;
          m.lim[rq.at][r] =
              none       ? 0
              : a.causal ? g.n - g.nq + (g.row0 + r) / shape.g + 1
                         : g.n;
          off |= none && r < g.rows;
        }
      }
      off = __any_sync(0xffffffffu, off);
      if (lane == 0) (&m.off[rq.at].x)[warp - 4] = off;
      asm volatile("cp.async.wait_all;" ::: "memory");
      // (a warp has four rows: its lanes go together)
#pragma unroll 1
      for (int r = r16; r < np; r += 16) {
        const uint4 u0 = *reinterpret_cast<const uint4*>(raw(r));
        const uint4 u1 = *reinterpret_cast<const uint4*>(raw(r) + 16);
        const uint32_t v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        float top = 0.f;                     // infinite: a NaN
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
        const int e = max((int)(__float_as_uint(top) >> 23) - 127, -119);
        float up = top < INFINITY ? __uint_as_float((134 - e) << 23)
                                  : __uint_as_float(0x7fffffffu);
        if (a.scale < 0.f) up = -up;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float2 y = make_float2(__uint_as_float(v[k] << 16) * up,
                                       __uint_as_float(v[k] & 0xffff0000u) * up);
          const uint32_t h =
              __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
          const float2 f = __half22float2(
              __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
          const uint32_t l = __nv_cvt_float2_to_fp8x2(
              make_float2((y.x - f.x) * 32.f, (y.y - f.y) * 32.f),
              __NV_SATFINITE, __NV_E4M3);
          if (k & 1) {
            hi[k >> 1] |= h << 16;
            lo[k >> 1] |= l << 16;
          } else {
            hi[k >> 1] = h;
            lo[k >> 1] = l;
          }
        }
        // (np is a multiple of 8: the second part's swizzle is the first's)
        uint8_t* dst = q + r * 128 + ((ch ^ (r & 7)) << 4);
        __syncwarp();
        *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(dst + np * 128) =
            make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (ch == 0)
          m.row[rq.at][r >> 1].rel[r & 1] =
              __uint_as_float(min(120 + kToRow + e, 254) << 23);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&m.q_full[rq.at]);
      rq.next();
    }
  } else if (warp >= 8) {
    // -------------------------------------------------------------- weights
    const int group = (warp - 8) >> 2, quarter = warp & 3;
    const int tok = quarter * 32 + lane;
    const uint32_t s_col =
        tmem + ((uint32_t)(quarter * 32) << 16) + group * PL::kColumns;
    const int page_bits = __ffs(a.page) - 1;
    Ring<2> rq;
    int tile = 0;                            // copied before the segment's
    uint32_t s_par = 0;
    bool ok = true;
    while (ok) {
      if (!next_segment()) break;
      const Segment g = m.seg[rg.at];
      done_segment();
      if (g.done) break;
      auto store = [&](int t, float sum) {
        const int at = g.tok0 + t * kTile + tok;
        if (at >= a.first && at < g.n) mass_store(a, g.b, g.hk, at, sum);
      };
      if (g.rows == 0) {                     // the sums are complete
        for (int t = group; t < g.T; t += kGroups) {
          store(t, m.keep[t][tok]);
          m.keep[t][tok] = 0.f;
        }
        continue;
      }
      const int np = (g.rows + 7) / 8 * 8;
      const Rows* rows = m.row[rq.at];
      const int* lims = m.lim[rq.at];
      ok = wait_for(&m.q_full[rq.at], rq.phase, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int4 o4 = m.off[rq.at];
      const bool off = (o4.x | o4.y | o4.z | o4.w) != 0;
#pragma unroll 1
      for (int t = group; t < g.T; t += kGroups) {
        ok = wait_for(&m.s_full[group], s_par, abort, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_par ^= 1;
        tc::fence_after_sync();
        const float ct = m.ks[(tile + t) % kStages][tok >> page_bits];
        const int at = g.tok0 + t * kTile + tok;
        // some row does not see all of the tile
        const bool masked = off || lims[0] < g.tok0 + (t + 1) * kTile;
        const uint64_t ct2 = pack2(ct, ct);
        const uint64_t rest2 = pack2(1.f / 32, 1.f / 32);
        uint64_t sum2[2] = {0, 0};
        // eight rows from c on, by pairs
        auto take = [&](int c, const float* hi, const float* lo) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const ulonglong2 r =
                *reinterpret_cast<const ulonglong2*>(&rows[(c + j) >> 1]);
            const uint64_t s2 = mul2(
                fma2(pack2(lo[j], lo[j + 1]), rest2, pack2(hi[j], hi[j + 1])),
                ct2);
            float x0, x1;
            unpack2(fma2(s2, r.x, r.y), x0, x1);
            if (masked) {
              if (at >= lims[c + j]) x0 = -INFINITY;
              if (at >= lims[c + j + 1]) x1 = -INFINITY;
            }
            sum2[j >> 1 & 1] =
                add2(sum2[j >> 1 & 1],
                     pack2(tc::ex2_approx(x0), tc::ex2_approx(x1)));
          }
        };
        int c = 0;
#pragma unroll 1
        for (; c + 16 <= np; c += 16) {
          float hi[16], lo[16];
          tmem_ld_x16(s_col + c, hi);
          tmem_ld_x16(s_col + np + c, lo);
          tmem_loaded(hi);
          tmem_loaded(lo);
          take(c, hi, lo);
          take(c + 8, hi + 8, lo + 8);
        }
        if (c < np) {
          float hi[8], lo[8];
          tmem_ld_x8(s_col + c, hi);
          tmem_ld_x8(s_col + np + c, lo);
          tmem_loaded(hi);
          tmem_loaded(lo);
          take(c, hi, lo);
        }
        float sum, sum_odd;
        unpack2(add2(sum2[0], sum2[1]), sum, sum_odd);
        sum += sum_odd;
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&m.s_empty[group]);
          tc::mbar_arrive(&m.k_empty[(tile + t) % kStages]);  // (the factors)
        }
        if (g.lone)
          store(t, sum);
        else
          m.keep[t][tok] += sum;
      }
      if (!ok) break;
      tile += g.T;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&m.q_empty[rq.at]);
      rq.next();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
  if (tid == 0 && m.abort) raise_error(a.err, kErrTimeout);
}

template <int kRows>
cudaError_t launch(const CUtensorMap& mk, const AttnMassArgs& a, const Shape& s,
                   int sms, cudaStream_t stream) {
  using PL = Plan<kRows>;
  auto* f = attn_mass_tc_kernel<kRows>;
  cudaError_t e = cudaFuncSetAttribute(
      f, cudaFuncAttributeMaxDynamicSharedMemorySize, PL::kSmem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3(sms), dim3(PL::kThreads), PL::kSmem, stream);
  return cudaLaunchKernelEx(&L.cfg, f, mk, a, s);
}

}  // namespace

cudaError_t launch_attn_mass_tc(const AttnMassArgs& a, int sms,
                                cudaStream_t stream) {
  Shape s;
  s.g = a.Hq / a.Hkv;
  s.first = a.first / kTile * kTile;
  const long long rows = (long long)a.Q * s.g;
  // (72 rows of 32 sequences: 73 us in one pass of 128, 94 in two of 40)
  s.rows = rows <= 64 ? 64 : kMaxRows;
  const long long tiles = (mass_most(a) - s.first + kTile - 1) / kTile;
  const long long passes = (rows + s.rows - 1) / s.rows;
  if ((long long)a.B * a.Hkv * (kUnitCost + tiles * passes) > 0x7fffffffll)
    return cudaErrorNotSupported;
  CUtensorMap mk;
  const uint64_t pool = (uint64_t)a.num_pages * a.Hkv * a.page;
  if (!make_tmap_u8_2d(&mk, a.k_codes, a.D, pool, 128, a.page))
    return cudaErrorInvalidValue;
  return s.rows == 64 ? launch<64>(mk, a, s, sms, stream)
                      : launch<kMaxRows>(mk, a, s, sms, stream);
}

}  // namespace dflash
