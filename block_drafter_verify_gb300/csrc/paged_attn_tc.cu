// Attention over the paged 8-bit cache on the tensor cores (tcgen05), for
// bf16 queries and heads of up to 128 dimensions.
//
// The cached codes go from HBM to the MMAs as they are: no kernel instruction
// touches a key or a value.  What has to meet them in 8 bits is the small
// side, split so that nothing is lost:
//   q    is scaled per row by a power of two and written as the sum of two
//        E4M3 numbers (8 bits, all that bf16 has); both products accumulate
//        into the same scores;
//   P    the softmax weights, rounded to fp16 (11 bits), are written as three
//        E4M3 numbers hi + mid / 16 + lo / 256, each with its own fp32
//        accumulator, so small weights keep bits below the range of one
//        E4M3 number.
// Scores are computed transposed: S^T[token, row] = K q^T and
// O^T[dim, row] = V^T P^T, so that the 128 lanes of an MMA are always full
// (tokens, then dimensions) and the number of (query, head) rows, a multiple
// of 16 up to 96, is the MMA's N: the cost follows the rows there are.  A
// thread of the softmax owns one token: its key's and its value's scale are
// one factor and one addend in the exponent (the value's scale, a power of
// two, rides on the weight).
//   V^T is the V tile as it lies (dimensions contiguous), an A operand with M
//   contiguous; P^T is written by token, 16 rows to a 16-byte unit, a B
//   operand with N contiguous.
// The running maximum is lazy: weights are taken against a reference that is
// raised (and the accumulators rescaled, by an exact power of two) only when
// a token beats it by more than 2^4.75; the pieces have room for that.
//
// Work is split by tiles of 128 tokens: all tiles of all (sequence, key head,
// row tile) units are numbered, and each CTA (one per SM) takes an equal run
// of them, whatever the sequences' lengths; a unit that is cut leaves partial
// sums that a second launch joins.
//
// Warps: 0 copies tiles (TMA, one box per page), 1 issues the MMAs, 2-3 lay
// out q, 4-11 do the softmax (two warps per lane quarter, half of the rows
// each) and write the output.  Every wait is bounded; on a timeout the CTA
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
constexpr int kThreads = 384;
constexpr int kUnitBytes = kTile * 128;  // a K or V tile in shared memory
constexpr int kSoftWarps = 8;
constexpr uint64_t kWait = 2000000000ull;  // 2 s
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kHead = 4.f;       // weights are 2^(score - ref + kHead)
constexpr float kRaise = 8.75f;    // 2^8.75 = 430 < 448

// Shared-memory plan for N rows.
template <int N>
struct Plan {
  static constexpr int Q = 2 * 2 * N * 128;       // two buffers, two parts
  static constexpr int P = 2 * 3 * N * 128;       // two buffers, three parts
  static constexpr int kFixed = 6 * 1024 + 1024;  // Meta, barriers, alignment
  static constexpr int kUnits = (232448 - Q - P - kFixed) / kUnitBytes;
  static constexpr int K = kUnits / 2 < 6 ? kUnits / 2 : 6;
  static constexpr int V = kUnits - K < 6 ? kUnits - K : 6;
  static constexpr int kBytes = kFixed + Q + P + (K + V) * kUnitBytes;
  static constexpr int kCols = 5 * N <= 128 ? 128 : 5 * N <= 256 ? 256 : 512;
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
  alignas(16) float back[kMaxRows];  // undoes the row's scaling
};

struct Meta {
  Segment seg[2];
  alignas(16) float neg_ref[kMaxRows], fac[kMaxRows], delta[kMaxRows];
  alignas(16) float warp_val[4][kMaxRows];
  float ct[6][8], lv[6][8];  // per V stage and page: key factor, log2 scale
  uint64_t kfull[6], kempty[6], vfull[6], vempty[6];
  uint64_t sfull[2], sempty[2], pfull[2], pvdone[2], qfull[2], qempty[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  long long start, count;    // first tile of this CTA's run and its length
  int b0;                    // its sequence, and the tiles before it there
  long long off0;
  long long warp_sum[kThreads / 32];
};
static_assert(sizeof(Meta) <= 6 * 1024, "");

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
  const int q0 = rt * s.N / s.g;
  if (q0 >= l.nq) return 0;
  int seen = l.n;
  if (a.causal) {
    const int q1 = min((min((rt + 1) * s.N, s.rows) - 1) / s.g, l.nq - 1);
    seen = max(0, min(l.n, l.n - l.nq + q1 + 1));
  }
  return (seen + kTile - 1) / kTile;
}
// Work of one key head of a sequence: its tiles, at least one per row tile.
__device__ __forceinline__ long long head_work(const PagedAttnArgs& a,
                                               const Shape& s, const Lens& l) {
  long long w = 0;
  for (int rt = 0; rt < s.row_tiles; ++rt) w += max(1, tiles_of(a, s, l, rt));
  return w;
}
// First tile of CTA c of the G that work (no more than there are tiles, so
// that each of them has one).
__device__ __forceinline__ long long run_start(long long total, int c, int G) {
  return c >= G ? total : total * c / G;
}

// Walks the units from a position in the numbering.
struct Walk {
  int b, hk, rt, tile;       // tile: first one not yet handed out
  long long left;            // tiles left in this CTA's run
  int first;                 // no segment handed out yet
};
__device__ void walk_start(const PagedAttnArgs& a, const Shape& s,
                           const Meta& m, Walk& w) {
  w.b = m.b0;
  w.left = m.count;
  w.first = 1;
  w.hk = w.rt = w.tile = 0;
  if (w.left <= 0) return;
  bool bad = false;
  const Lens l = lens_of(a, w.b, &bad);
  const long long h = head_work(a, s, l);
  long long o = m.off0;
  w.hk = (int)(o / h);
  o -= w.hk * h;
  for (;; ++w.rt) {
    const int t = max(1, tiles_of(a, s, l, w.rt));
    if (o < t) break;
    o -= t;
  }
  w.tile = (int)o;
}
struct Part {
  int b, hk, rt, t0, t1, whole, first;
  Lens l;
};
// The next segment; false at the end of the run.
__device__ bool walk_next(const PagedAttnArgs& a, const Shape& s, Walk& w,
                          Part& p) {
  if (w.left <= 0) return false;
  bool bad = false;
  p.l = lens_of(a, w.b, &bad);
  const int t = tiles_of(a, s, p.l, w.rt);
  const int work = max(1, t);
  const int take = (int)min((long long)(work - w.tile), w.left);
  p.b = w.b;
  p.hk = w.hk;
  p.rt = w.rt;
  p.t0 = w.tile;
  p.t1 = min(t, w.tile + take);
  p.whole = take == work;
  p.first = w.first;
  w.first = 0;
  w.left -= take;
  w.tile += take;
  if (w.tile == work) {
    w.tile = 0;
    if (++w.rt == s.row_tiles) {
      w.rt = 0;
      if (++w.hk == a.Hkv) {
        w.hk = 0;
        ++w.b;
      }
    }
  }
  return true;
}

// ---- PTX ------------------------------------------------------------------
// Instruction descriptor: E4M3 x E4M3 -> fp32; both operands with M / N
// contiguous (bits 15, 16) for the second product.
__host__ __device__ constexpr uint32_t idesc_mn(int N) {
  return tc::idesc_e4m3_f32(128, N) | (1u << 15) | (1u << 16);
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
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}"
      ", [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8};" ::"r"(addr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
      "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
      : "memory");
}
// Wait for this thread's TMEM loads; no use of v is scheduled before it.
template <int M>
__device__ __forceinline__ void tmem_loaded(float (&v)[M]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < M; ++i) asm volatile("" : "+f"(v[i])::"memory");
}
__device__ __forceinline__ void tmem_stored() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Barrier of 128 threads; true if `p` is true in any of them.
__device__ __forceinline__ bool half_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void half_sync(int id) {
  asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(id) : "memory");
}

// Two weights (fp32, at most 430) as three pairs of codes.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi,
                                       uint32_t& mid, uint32_t& lo) {
  const __half2 up = __float2half2_rn(16.f), dn = __float2half2_rn(-16.f);
  const __half2 y = __floats2half2_rn(a, b);
  hi = __nv_cvt_halfraw2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  const __half2 h1(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3));
  const __half2 r1 = __hfma2(h1, dn, __hmul2(y, up));  // 16 (y - hi), exact
  mid = __nv_cvt_halfraw2_to_fp8x2(r1, __NV_SATFINITE, __NV_E4M3);
  const __half2 h2(__nv_cvt_fp8x2_to_halfraw2(mid, __NV_E4M3));
  const __half2 r2 = __hfma2(h2, dn, __hmul2(r1, up));
  lo = __nv_cvt_halfraw2_to_fp8x2(r2, __NV_SATFINITE, __NV_E4M3);
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ PagedAttnArgs a,
                         const Shape shape, float* __restrict__ part) {
  using PL = Plan<N>;
  constexpr int HR = N / 2;  // rows of a softmax warp
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sk = base;
  uint8_t* sv = sk + PL::K * kUnitBytes;
  uint8_t* sq = sv + PL::V * kUnitBytes;   // [2][2][N][128]
  uint8_t* sp = sq + PL::Q;                // [2][3][N / 16][128][16]
  Meta& m = *reinterpret_cast<Meta*>(sp + PL::P);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort = &m.abort;

  if (tid == 0) {
    for (int i = 0; i < 6; ++i) {
      tc::mbar_init(&m.kfull[i], 1);
      tc::mbar_init(&m.kempty[i], 1);
      tc::mbar_init(&m.vfull[i], 1);
      tc::mbar_init(&m.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&m.sfull[i], 1);
      tc::mbar_init(&m.sempty[i], kSoftWarps);
      tc::mbar_init(&m.pfull[i], kSoftWarps);
      tc::mbar_init(&m.pvdone[i], 1);
      tc::mbar_init(&m.qfull[i], 2);
      tc::mbar_init(&m.qempty[i], 1 + kSoftWarps);
    }
    tc::mbar_init(&m.drain, 1);
    m.abort = 0;
    m.b0 = 0;
    m.off0 = 0;
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
  pdl_trigger();
  pdl_wait();
  // ---- where this CTA's run of tiles starts ------------------------------
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long w = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b)
      w += a.Hkv * head_work(a, shape, lens_of(a, b, &bad));
    if (bad && blockIdx.x == 0) raise_error(a.err, kErrBadIndex);
    long long run = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (lane == 31) m.warp_sum[warp] = run;
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) run += m.warp_sum[i];
      total += m.warp_sum[i];
    }
    const int G = (int)min((long long)gridDim.x, total);
    const long long p0 = run_start(total, blockIdx.x, G);
    const long long p1 = run_start(total, blockIdx.x + 1, G);
    if (tid == 0) {
      m.start = p0;
      m.count = p1 - p0;
    }
    if (p1 > p0 && p0 >= run - w && p0 < run) {
      long long o = p0 - (run - w);
      int b = b0;
      for (; b < b1; ++b) {
        const long long v = a.Hkv * head_work(a, shape, lens_of(a, b, &bad));
        if (o < v) break;
        o -= v;
      }
      m.b0 = b;
      m.off0 = o;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = m.tmem;

  if (warp == 0) {
    // ---------------------------------------------------------- producer
    Walk w;
    walk_start(a, shape, m, w);
    Part p;
    const int pt = kTile / a.page;         // pages of a tile
    const int oob = a.num_pages * a.Hkv * a.page;  // a row past the pool
    const uint32_t box = (uint32_t)a.page * 128;
    const float c = a.scale * kLog2e;
    long long i = 0, nk = 0, nv = 0;       // tiles, K and V copies so far
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
      float ks = load_scale(a.k_scale, id), vs = load_scale(a.v_scale, id);
      float ks1 = load_scale(a.k_scale, id1), vs1 = load_scale(a.v_scale, id1);
      for (int t = p.t0; t < p.t1; ++t, ++i) {
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
        const float pk = __shfl_sync(0xffffffffu, ks, from & 31);
        const float pv = __shfl_sync(0xffffffffu, vs, from & 31);
        const bool have = lane < pt && t * pt + lane < pages;
        const bool bad = have && (pid < 0 || pid >= a.num_pages);
        if (bad) raise_error(a.err, kErrBadIndex);
        const int row = bad ? oob : (pid * a.Hkv + p.hk) * a.page;
        const uint32_t bytes = box * __popc(__ballot_sync(0xffffffffu, have));
        const int kst = (int)(i % PL::K), vst = (int)(i % PL::V);
        ok = tc::mbar_wait_bounded(&m.kempty[kst],
                                   (uint32_t)((i / PL::K) & 1) ^ 1, abort,
                                   kWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(&m.kfull[kst], bytes);
        __syncwarp();
        if (have)
          tc::tma_load_2d(sk + kst * kUnitBytes + lane * box, &map_k,
                          &m.kfull[kst], 0, row);
        ++nk;
        ok = tc::mbar_wait_bounded(&m.vempty[vst],
                                   (uint32_t)((i / PL::V) & 1) ^ 1, abort,
                                   kWait);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane < pt) {
          m.ct[vst][lane] = have && !bad ? pk * c : 0.f;
          m.lv[vst][lane] = have ? log2f(fmaxf(pv, 0x1p-100f)) : 0.f;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect_tx(&m.vfull[vst], bytes);
        __syncwarp();
        if (have)
          tc::tma_load_2d(sv + vst * kUnitBytes + lane * box, &map_v,
                          &m.vfull[vst], 0, row);
        ++nv;
      }
    }
    // no copy is in flight when the CTA leaves, whatever the others did
    int never = 0;
    for (long long j = max(0ll, nk - PL::K); j < nk; ++j)
      tc::mbar_wait_bounded(&m.kfull[j % PL::K], (uint32_t)((j / PL::K) & 1),
                            &never, kWait);
    for (long long j = max(0ll, nv - PL::V); j < nv; ++j)
      tc::mbar_wait_bounded(&m.vfull[j % PL::V], (uint32_t)((j / PL::V) & 1),
                            &never, kWait);
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t id_s = tc::idesc_e4m3_f32(128, N);
      constexpr uint32_t id_o = idesc_mn(N);
      const uint32_t o_col = tmem + 2 * N;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        ok = ok && tc::mbar_wait_bounded(bar, par, abort, kWait);
        return ok;
      };
      long long i = 0;
      for (int s = 0; ok; ++s) {
        const int qb = s & 1;
        if (!wait(&m.qfull[qb], (s >> 1) & 1)) break;
        const Segment& g = m.seg[qb];
        if (g.done) break;
        const int T = g.t1 - g.t0;
        const uint32_t q0 = tc::smem_u32(sq) + qb * 2 * N * 128;
        auto scores = [&](long long j) {
          const int st = (int)(j % PL::K), sb = (int)(j & 1);
          if (!wait(&m.kfull[st], (uint32_t)((j / PL::K) & 1))) return;
          if (!wait(&m.sempty[sb], (uint32_t)((j >> 1) & 1) ^ 1)) return;
          tc::fence_after_sync();
          const uint32_t k0 = tc::smem_u32(sk) + st * kUnitBytes;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_e4m3(tmem + sb * N, tc::sdesc_k_sw128(k0 + 32 * k),
                           tc::sdesc_k_sw128(q0 + h * N * 128 + 32 * k), id_s,
                           (h | k) != 0);
          tc::mma_commit(&m.kempty[st]);
          tc::mma_commit(&m.sfull[sb]);
        };
        if (T > 0) scores(i);
        for (int t = 0; ok && t < T; ++t, ++i) {
          if (t + 1 < T) scores(i + 1);
          const int st = (int)(i % PL::V), sb = (int)(i & 1);
          if (!wait(&m.vfull[st], (uint32_t)((i / PL::V) & 1))) break;
          if (!wait(&m.pfull[sb], (uint32_t)((i >> 1) & 1))) break;
          tc::fence_after_sync();
          const uint32_t v0 = tc::smem_u32(sv) + st * kUnitBytes;
          const uint32_t p0 = tc::smem_u32(sp) + sb * 3 * N * 128;
#pragma unroll
          for (int h = 0; h < 3; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_e4m3(o_col + h * N, sdesc_mn_sw128(v0 + 4096 * k),
                           sdesc_mn_plain(p0 + h * N * 128 + 512 * k), id_o,
                           t > 0 || k > 0);
          tc::mma_commit(&m.vempty[st]);
          tc::mma_commit(&m.pvdone[sb]);
        }
        if (ok) tc::mma_commit(&m.qempty[qb]);
      }
      tc::mma_commit(&m.drain);
      int never = 0;
      tc::mbar_wait_bounded(&m.drain, 0, &never, kWait);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------ layout of q
    Walk w;
    walk_start(a, shape, m, w);
    const int qt = tid - 64;               // 0..63
    const int ch = qt & 7;                 // 16 dimensions of a row
    for (int s = 0;; ++s) {
      const int qb = s & 1;
      bool ok = tc::mbar_wait_bounded(&m.qempty[qb],
                                      (uint32_t)((s >> 1) & 1) ^ 1, abort,
                                      kWait);
      if (!__all_sync(0xffffffffu, ok)) break;
      Segment& g = m.seg[qb];
      Part p;
      const bool more = walk_next(a, shape, w, p);
      if (more) {
        const int row0 = p.rt * N;
        uint8_t* q0 = sq + qb * 2 * N * 128;
        for (int r = qt >> 3; r < N; r += 8) {
          const int row = row0 + r;
          const int qi = row / shape.g;
          const bool live = row < shape.rows && qi < p.l.nq;
          float x[16];
          float big = 0.f;
          if (live && ch * 16 < a.D) {
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) +
                (((size_t)p.b * a.Q + qi) * a.Hq + p.hk * shape.g +
                 row % shape.g) * a.D + ch * 16);
            const uint4 u[2] = {src[0], src[1]};
            const uint32_t* v = reinterpret_cast<const uint32_t*>(u);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              x[2 * k] = __uint_as_float(v[k] << 16);
              x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              big = x[k] == x[k] ? fmaxf(big, fabsf(x[k])) : INFINITY;
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = 0.f;
          }
#pragma unroll
          for (int o = 4; o; o >>= 1)
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          // the row's largest value to [128, 256)
          const int e = max((int)(__float_as_uint(big) >> 23) - 127, -100);
          const float up = big < INFINITY ? __uint_as_float((134 - e) << 23)
                                          : __uint_as_float(0x7fffffffu);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 y = make_float2(x[2 * k] * up, x[2 * k + 1] * up);
            const uint32_t h =
                __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            const float2 f = __half22float2(
                __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3)));
            const uint32_t l = __nv_cvt_float2_to_fp8x2(
                make_float2(y.x - f.x, y.y - f.y), __NV_SATFINITE, __NV_E4M3);
            if (k & 1) {
              hi[k >> 1] |= h << 16;
              lo[k >> 1] |= l << 16;
            } else {
              hi[k >> 1] = h;
              lo[k >> 1] = l;
            }
          }
          uint8_t* dst = q0 + r * 128 + ((ch ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) =
              make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + N * 128) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (ch == 0) {
            g.back[r] = __uint_as_float((120 + e) << 23);  // 2^(e - 7)
            g.lim[r] = !live      ? 0x7fffffff
                       : a.causal ? min(p.l.n, p.l.n - p.l.nq + qi + 1)
                                  : p.l.n;
          }
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
          g.min_lim = a.causal ? min(p.l.n, p.l.n - p.l.nq +
                                                row0 / shape.g + 1)
                               : p.l.n;
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
    const int half = (warp - 4) >> 2, quarter = warp & 3;
    const int ht = tid - 128 - half * 128;  // thread of the half
    const int tok = quarter * 32 + lane;
    const int rb = half * HR;
    const int bar = 1 + half;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_col = lanes + 2 * N + rb;
    long long i = 0;
    bool live = true;
    for (int s = 0; live; ++s) {
      const int qb = s & 1;
      bool ok = tc::mbar_wait_bounded(&m.qfull[qb], (s >> 1) & 1, abort,
                                      kWait);
      if (half_any(bar, !ok)) break;
      const Segment& g = m.seg[qb];
      if (g.done) break;
      const int T = g.t1 - g.t0;
      float l[HR];
#pragma unroll
      for (int r = 0; r < HR; ++r) l[r] = 0.f;
      if (ht < HR) m.neg_ref[rb + ht] = 0.f;
      half_sync(bar);
      float lv_ref = 0.f;
      for (int t = 0; t < T; ++t, ++i) {
        const int sb = (int)(i & 1), st = (int)(i % PL::V);
        ok = tc::mbar_wait_bounded(&m.sfull[sb], (uint32_t)((i >> 1) & 1),
                                   abort, kWait) &&
             tc::mbar_wait_bounded(&m.vfull[st], (uint32_t)((i / PL::V) & 1),
                                   abort, kWait);
        ok = __all_sync(0xffffffffu, ok);
        float y[HR];
        if (ok) {
          tc::fence_after_sync();
#pragma unroll
          for (int r = 0; r < HR; r += 8)
            tmem_ld8(lanes + sb * N + rb + r, y + r);
          tmem_loaded(y);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&m.sempty[sb]);
        } else {
#pragma unroll
          for (int r = 0; r < HR; ++r) y[r] = 0.f;
        }
        const int pos = (g.t0 + t) * kTile + tok;
        const float ct = m.ct[st][tok / a.page], lv = m.lv[st][tok / a.page];
        if (t == 0) lv_ref = m.lv[st][0];
        const float fl = tc::ex2_approx(fminf(lv_ref - lv, 100.f));
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          const float4 bk = *reinterpret_cast<const float4*>(&g.back[rb + r]);
          const float4 nr =
              *reinterpret_cast<const float4*>(&m.neg_ref[rb + r]);
          y[r] = fmaf(y[r] * bk.x, ct, lv) + nr.x;
          y[r + 1] = fmaf(y[r + 1] * bk.y, ct, lv) + nr.y;
          y[r + 2] = fmaf(y[r + 2] * bk.z, ct, lv) + nr.z;
          y[r + 3] = fmaf(y[r + 3] * bk.w, ct, lv) + nr.w;
        }
        if ((g.t0 + t + 1) * kTile > g.min_lim) {
#pragma unroll
          for (int r = 0; r < HR; ++r)
            y[r] = pos < min(g.lim[rb + r], g.n) ? y[r] : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < HR; ++r) top = fmaxf(top, y[r]);
        if (half_any(bar, t == 0 || top > kRaise || !ok)) {
          // ---- raise the references -------------------------------------
          if (half_any(bar, !ok)) { live = false; break; }
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            const float z = warp_max(y[r]);
            if (lane == 0) m.warp_val[quarter][rb + r] = z;
          }
          half_sync(bar);
          if (ht < HR) {
            const int r = rb + ht;
            float z = fmaxf(fmaxf(m.warp_val[0][r], m.warp_val[1][r]),
                            fmaxf(m.warp_val[2][r], m.warp_val[3][r]));
            // y = score + neg_ref, neg_ref = kHead - ref (0 before the
            // first tile and for a row that sees nothing)
            float d = 0.f;
            if (z > -INFINITY && (t == 0 || z > kHead)) d = kHead - ceilf(z);
            m.delta[r] = d;
            m.fac[r] = tc::ex2_approx(d);
            m.neg_ref[r] += d;
          }
          half_sync(bar);
          if (t > 0) {
            ok = tc::mbar_wait_bounded(&m.pvdone[sb ^ 1],
                                       (uint32_t)(((i - 1) >> 1) & 1), abort,
                                       kWait);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();
#pragma unroll
            for (int r = 0; r < HR; r += 8) {
              float f[8];
              bool one = true;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                f[k] = m.fac[rb + r + k];
                one &= f[k] == 1.f;
                l[r + k] *= f[k];
              }
              if (!one && ok) {
#pragma unroll
                for (int h = 0; h < 3; ++h) {
                  float o[8];
                  tmem_ld8(o_col + h * N + r, o);
                  tmem_loaded(o);
#pragma unroll
                  for (int k = 0; k < 8; ++k) o[k] *= f[k];
                  tmem_st8(o_col + h * N + r, o);
                }
              }
            }
            tmem_stored();
            tc::fence_before_sync();
          }
#pragma unroll
          for (int r = 0; r < HR; ++r) y[r] += m.delta[rb + r];
        }
        // ---- the weights, in three parts -----------------------------------
        ok = tc::mbar_wait_bounded(&m.pvdone[sb], (uint32_t)((i >> 1) & 1) ^ 1,
                                   abort, kWait);
        ok = __all_sync(0xffffffffu, ok);
        uint8_t* dst = sp + sb * 3 * N * 128 + tok * 16;
#pragma unroll
        for (int r = 0; r < HR; r += 8) {
          uint32_t c[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e0 = tc::ex2_approx(y[r + 2 * k]);
            const float e1 = tc::ex2_approx(y[r + 2 * k + 1]);
            l[r + 2 * k] = fmaf(e0, fl, l[r + 2 * k]);
            l[r + 2 * k + 1] = fmaf(e1, fl, l[r + 2 * k + 1]);
            split3(e0, e1, c[0][k], c[1][k], c[2][k]);
          }
          if (ok) {
            const int row = rb + r;
#pragma unroll
            for (int h = 0; h < 3; ++h)
              *reinterpret_cast<uint2*>(dst + h * N * 128 +
                                        (row >> 4) * 2048 + (row & 8)) =
                  make_uint2(c[h][0] | c[h][1] << 16, c[h][2] | c[h][3] << 16);
          }
        }
        if (half == 0 && pos >= g.n && ok) {
          // values past the cache's end may be anything: their weight is 0
          uint4* v = reinterpret_cast<uint4*>(sv + st * kUnitBytes + tok * 128);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = make_uint4(0, 0, 0, 0);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&m.pfull[sb]);
      }
      if (!live) break;
      // ---- the segment's result ------------------------------------------
      if (T > 0) {
        ok = tc::mbar_wait_bounded(&m.pvdone[(i - 1) & 1],
                                   (uint32_t)(((i - 1) >> 1) & 1), abort,
                                   kWait);
        if (half_any(bar, !ok)) break;
        tc::fence_after_sync();
      }
#pragma unroll
      for (int r = 0; r < HR; ++r) {
        const float v = warp_sum(l[r]);
        if (lane == 0) m.warp_val[quarter][rb + r] = v;
      }
      half_sync(bar);
      const float lift = exp2f(lv_ref);
      if (ht < HR) {
        const int r = rb + ht, row = g.row0 + r;
        const float sum = (m.warp_val[0][r] + m.warp_val[1][r]) +
                          (m.warp_val[2][r] + m.warp_val[3][r]);
        const float ref = -m.neg_ref[r] - lv_ref;   // log2 of what sum counts
        const int qi = row / shape.g;
        const bool seen = sum > 0.f || sum != sum;  // a NaN stays one
        if (g.whole) {
          const bool on = seen && row < shape.rows && qi < g.nq;
          m.fac[r] = on ? lift / sum : 0.f;
          if (row < shape.rows && a.lse)
            a.lse[((size_t)g.b * a.Q + qi) * a.Hq + g.hk * shape.g +
                  row % shape.g] =
                on ? (log2f(sum) + ref) * 0.6931471805599453f : -INFINITY;
        } else {
          m.fac[r] = lift;
          float2* ml = reinterpret_cast<float2*>(
              part + (size_t)2 * gridDim.x * N * 128);
          ml[(size_t)g.slot * N + r] =
              make_float2(seen ? ref : -INFINITY, seen ? sum : 0.f);
        }
      }
      half_sync(bar);
      const int d = tok;
#pragma unroll
      for (int r = 0; r < HR; r += 8) {
        float o[24];
        if (T > 0) {
#pragma unroll
          for (int h = 0; h < 3; ++h) tmem_ld8(o_col + h * N + r, o + 8 * h);
          tmem_loaded(o);
        } else {
#pragma unroll
          for (int k = 0; k < 24; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float f = m.fac[rb + r + k];
          const float v =
              fmaf(o[16 + k], 0x1p-8f, fmaf(o[8 + k], 0x1p-4f, o[k])) * f;
          const int row = g.row0 + rb + r + k;
          if (g.whole) {
            if (row < shape.rows && d < a.D) {
              const int qi = row / shape.g;
              static_cast<__nv_bfloat16*>(a.out)[
                  (((size_t)g.b * a.Q + qi) * a.Hq + g.hk * shape.g +
                   row % shape.g) * a.D + d] =
                  __float2bfloat16_rn(f == 0.f ? 0.f : v);
            }
          } else {
            part[((size_t)g.slot * N + rb + r + k) * 128 + d] = v;
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&m.qempty[qb]);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, PL::kCols);
  if (tid == 0 && m.abort) raise_error(a.err, kErrTimeout);
}

// Joins the partial sums of the units that the runs cut: 128 threads (one
// per dimension) for up to eight rows of a unit.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(128)
    paged_attn_tc_join_kernel(const __grid_constant__ PagedAttnArgs a,
                              const Shape shape, int grid,
                              const float* __restrict__ part) {
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  int u = blockIdx.x;
  const int rt = u % shape.row_tiles;
  u /= shape.row_tiles;
  const int hk = u % a.Hkv, b = u / a.Hkv;
  // tiles before this unit, and all tiles
  long long before = 0, total = 0;
  bool bad = false;
  for (int i = tid; i < a.B; i += 128) {
    const long long w = a.Hkv * head_work(a, shape, lens_of(a, i, &bad));
    total += w;
    if (i < b) before += w;
  }
  __shared__ long long s_sum[2][4];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    s_sum[0][tid >> 5] = before;
    s_sum[1][tid >> 5] = total;
  }
  __syncthreads();
  before = s_sum[0][0] + s_sum[0][1] + s_sum[0][2] + s_sum[0][3];
  total = s_sum[1][0] + s_sum[1][1] + s_sum[1][2] + s_sum[1][3];
  const int G = (int)min((long long)grid, total);
  const Lens l = lens_of(a, b, &bad);
  before += hk * head_work(a, shape, l);
  for (int i = 0; i < rt; ++i) before += max(1, tiles_of(a, shape, l, i));
  const long long end = before + max(1, tiles_of(a, shape, l, rt));
  const int c0 = (int)(((before + 1) * G - 1) / total);
  const int c1 = (int)((end * G - 1) / total);  // of the last tile, end - 1
  if (c0 == c1) return;
  const int n = c1 - c0 + 1;
  auto slot = [&](int i) {
    const int c = c0 + i;
    return 2 * c + (i == 0 && run_start(total, c, G) != before ? 1 : 0);
  };
  const float2* ml = reinterpret_cast<const float2*>(
      part + (size_t)2 * grid * shape.N * 128);
  __shared__ float s_w[kMaxCtas];
  const int r1 = min(shape.N, (int)(blockIdx.y + 1) * kJoinRows);
  for (int r = blockIdx.y * kJoinRows; r < r1; ++r) {
    const int row = rt * shape.N + r;
    if (row >= shape.rows) break;
    __syncthreads();
    if (tid < 32) {
      float top = -INFINITY;
      for (int i = lane; i < n; i += 32)
        top = fmaxf(top, ml[(size_t)slot(i) * shape.N + r].x);
      top = warp_max(top);
      float sum = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float2 v = ml[(size_t)slot(i) * shape.N + r];
        const float w = v.x == -INFINITY ? 0.f : exp2f(v.x - top);
        s_w[i] = w;
        sum += w * v.y;
      }
      sum = warp_sum(sum);
      const int qi = row / shape.g;
      const bool on = (sum > 0.f || sum != sum) && qi < l.nq;
      const float inv = on ? 1.f / sum : 0.f;
      for (int i = lane; i < n; i += 32) s_w[i] *= inv;
      if (lane == 0 && a.lse)
        a.lse[((size_t)b * a.Q + qi) * a.Hq + hk * shape.g + row % shape.g] =
            on ? (log2f(sum) + top) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();
    if (tid < a.D) {
      float o = 0.f;
#pragma unroll 4
      for (int i = 0; i < n; ++i)
        o = fmaf(s_w[i], part[((size_t)slot(i) * shape.N + r) * 128 + tid], o);
      static_cast<__nv_bfloat16*>(a.out)[
          (((size_t)b * a.Q + row / shape.g) * a.Hq + hk * shape.g +
           row % shape.g) * a.D + tid] = __float2bfloat16_rn(o);
    }
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
  PdlLaunch L(dim3(G), dim3(kThreads), Plan<N>::kBytes, stream);
  return cudaLaunchKernelEx(&L.cfg, f, mk, mv, a, s, part);
}

}  // namespace

bool paged_attn_tc_takes(int D, dflash_dtype dt) {
  return dt == DFLASH_BF16 && D <= 128;
}

size_t paged_attn_tc_ws(int B, int Q, int Hq, int Hkv) {
  (void)B;
  const Shape s = shape_of(Q, Hq, Hkv);
  return (size_t)2 * kMaxCtas * s.N * (128 + 2) * sizeof(float);
}

cudaError_t launch_paged_attn_tc(const PagedAttnArgs& a, int sms, float* part,
                                 cudaStream_t stream) {
  const Shape s = shape_of(a.Q, a.Hq, a.Hkv);
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
  const long long units = (long long)a.B * a.Hkv * s.row_tiles;
  if (units > 0x7fffffffll) return cudaErrorInvalidValue;
  const int most = std::min(s.N, s.rows);
  PdlLaunch J(dim3((unsigned)units, (most + kJoinRows - 1) / kJoinRows),
              dim3(128), 0, stream);
  return cudaLaunchKernelEx(&J.cfg, paged_attn_tc_join_kernel, a, s, G,
                            (const float*)part);
}

}  // namespace dflash
