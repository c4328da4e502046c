// Sampling with temperature, top-k, top-p and min-p from given uniforms, and
// the filtered logits for the lossless verify.
//
// Mathematics.  Tokens are ranked by (logit descending, id ascending); every
// filter keeps a prefix of that ranking, so together they keep the tokens
// not below one cut.  The cut is a 64-bit word: the logit's order-preserving
// 32-bit key over the complement of the id.  Weights are 64-bit integers
// floor(exp(.) 2^44): their sums are exact, so the cut, the totals and the
// drawn token do not depend on how the row is split over threads and CTAs.
//
// A cluster of CTAs owns a row: each CTA reads its slice from HBM once and
// keeps it in shared memory (by bulk copies: more bytes in flight than its
// threads could have), where all later passes run; only maxima, histograms,
// short lists and sums travel between the CTAs (distributed shared memory).
// What happens then is the row's own:
//   T = 0           the first maximum;
//   top-k           the k-th largest of the threads' own maxima bounds the
//                   k-th largest token from below, so one comparison per
//                   token gathers few more than k candidates (with small k
//                   each CTA takes its own bound, which spares two cluster
//                   barriers); one CTA sorts them, applies top-p and min-p,
//                   and draws among them;
//   top-p only      a histogram of weights over bins of (max - l) / T finds
//                   the bin in which the weight passes p W, whose members are
//                   gathered and sorted; kept weights by warp chunk, the draw;
//   neither         kept weights by warp chunk, the draw.
// What overflows a list (ties by the thousand, a tail of weightless tokens)
// is resolved by radix selection on the 64-bit words instead.
#include <cooperative_groups.h>

#include <algorithm>

#include "kernels.h"
#include "tc_ptx.cuh"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr float kBinsPerUnit = 32.f;   // bins of 1/32 in (max - l) / T
constexpr int kCand = 2048;            // candidates, over the cluster
constexpr int kOwnBound = 128;         // largest k for a bound of each CTA
constexpr int kChunks = 4;             // copies of a slice
constexpr uint64_t kWait = 2000000000ull;  // 2 s
constexpr int kCandBins = 512;         // bins of 1/16 for their bound
constexpr int kList = 256;             // members of one bin
constexpr int kCollects = 3;           // lists that a row may gather
constexpr int kMaxCluster = 8;

struct SampleArgs {
  const void* logits;
  long long ld;
  const float* temperature;
  const int* top_k;
  const float *top_p, *min_p, *u;
  int R, V, slice;   // slice: tokens per CTA, a multiple of 8
  int resident;      // the slice fits in shared memory
  int* token;
  int* n_kept;
  float* filtered;
  int* err;
};

// Order-preserving key of a logit (equal for -0 and 0); 0 is below -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t w = __float_as_uint(x + 0.f);
  return w & 0x80000000u ? ~w : w | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // key_of(-inf)

__device__ __forceinline__ u64 word_of(float x, int id) {
  return (u64)key_of(x) << 32 | (uint32_t)~id;
}

template <typename U>
__device__ __forceinline__ U warp_total(U v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
struct Shared {
  // written by this CTA, read by the cluster
  float top;             // largest logit of the slice
  int first;             // T = 0: first token of the slice that has it
  u64 total;             // weight of the slice
  u64 kept_w[kWarps];    // kept weight of each warp's chunk
  float kept_least[kWarps];  // and its smallest kept logit
  uint32_t kept_n;
  uint32_t odd;          // a logit of the slice is not finite
  uint32_t lists[kCollects][kMaxCluster];  // lengths of every CTA's lists
  uint32_t row_listed[kCollects];  // the first CTA's: places taken in all_cand
  uint64_t landed[kChunks];  // barriers of the slice's copies
  // this CTA's own
  uint32_t listed;
  uint32_t list_at;      // place of its list among the row's
  uint32_t n_list;       // members of a bin
  uint32_t least_key;
  u64 target;            // what the weight in found_bin reaches
  float t, top_p, min_p, u;
  int top_k;
  u64 warp_w[kWarps];
  uint32_t warp_n[kWarps];
  int found_bin;
  u64 found_w;           // weight before the found bin
  uint32_t found_n;      // tokens before it
  u64 cut;
  u64 kept_before;       // weight of the tokens down to the cut
  int kept;
  union {
    struct {
      uint32_t count[kBins];              // read by the cluster
      uint32_t w_lo[kBins], w_hi[kBins];  // read by the cluster
      union {
        uint32_t all_count[kBins];
        struct {
          u64 list[kList], list_w[kList];
        };
      };
      u64 all_w[kBins];
    };
    struct {
      u64 cand[kCand];      // this CTA's candidates
      u64 all_cand[kCand];  // the row's, in the first CTA
    };
  };
};

// What a row's weights are made from.
struct Row {
  float top, inv_t;
  bool greedy;
};
__device__ __forceinline__ float x_of(float l, const Row& r) {
  if (l == r.top) return 1.f;  // also where the difference is no number
  return expf(__fmul_rn(__fsub_rn(l, r.top), r.inv_t));
}
// The same where the maximum and 1 / T are finite and l is a number.
__device__ __forceinline__ float x_plain(float l, const Row& r) {
  return expf(__fmul_rn(__fsub_rn(l, r.top), r.inv_t));
}
// floor(x 2^44) for 0 <= x <= 1, as 21 and 23 bits that additions to 2^23
// (whose last place is 1) round off towards zero: the conversion to a 64-bit
// integer has a sixteenth of their rate.
struct WeightBits {
  uint32_t hi, lo;  // 0x4b000000 (the bits of 2^23) above the halves
};
__device__ __forceinline__ WeightBits weight_bits(float x) {
  const float xs = __fmul_rn(x, 0x1p21f);
  const float hi = __fadd_rz(xs, 0x1p23f);
  const float rest = __fsub_rn(xs, __fsub_rn(hi, 0x1p23f));  // exact
  const float lo = __fmaf_rz(rest, 0x1p23f, 0x1p23f);
  return WeightBits{__float_as_uint(hi), __float_as_uint(lo)};
}
__device__ __forceinline__ u64 weight_of(float x) {
  const WeightBits w = weight_bits(x);
  return (u64)(w.hi - 0x4b000000u) * (1u << 23) + (w.lo - 0x4b000000u);
}
// Bin of a logit: 0 at the maximum, rising as it falls; monotone in l.
__device__ __forceinline__ int bin_of(float l, const Row& r) {
  if (l == r.top) return 0;
  const float z = __fmul_rn(__fmul_rn(__fsub_rn(r.top, l), r.inv_t),
                            kBinsPerUnit);
  return z < (float)(kBins - 1) ? (int)z : kBins - 1;
}

// A logit below all of bins 0 .. bin (-inf after the last): z is less than
// (bin + 1) / kBinsPerUnit there, with room for its roundings.
__device__ __forceinline__ float bin_floor(int bin, const Row& r, float t) {
  if (bin >= kBins - 1) return -INFINITY;
  const float z = (float)(bin + 1) / kBinsPerUnit;
  return r.top - z * t * 1.0001f - fabsf(r.top) * 1e-6f;
}

// A logit above all of bins bin, bin + 1, ...
__device__ __forceinline__ float bin_ceil(int bin, const Row& r, float t) {
  const float z = (float)bin / kBinsPerUnit;
  return r.top - z * t * 0.9999f + fabsf(r.top) * 1e-6f;
}

__device__ __forceinline__ void add_weight(Shared& S, int bin, u64 w) {
  const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
  const uint32_t old = atomicAdd(&S.w_lo[bin], lo);
  const uint32_t up = hi + (old + lo < old ? 1u : 0u);
  if (up) atomicAdd(&S.w_hi[bin], up);
}

// Sums the cluster's histograms (first n bins) into all_count, all_w of
// every CTA.  Cluster barriers on both sides: the histograms are complete
// before, and may be cleared after.
__device__ void reduce_bins(Shared& S, cg::cluster_group& cl, int n) {
  cl.sync();
  const int C = cl.num_blocks();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint32_t c = 0;
    u64 w = 0;
    for (int r = 0; r < C; ++r) {
      const Shared* o = cl.map_shared_rank(&S, r);
      c += o->count[i];
      w += (u64)o->w_hi[i] << 32 | 0u;
      w += o->w_lo[i];
    }
    S.all_count[i] = c;
    S.all_w[i] = w;
  }
  cl.sync();
}

// The first of n bins at which the running count reaches `need_n` (by_weight
// false) or the running weight reaches need_w(weight of all bins); its
// predecessors' sums.  found_bin = -1 if none does.  Whole CTA, which has left
// the last call's results behind.
template <typename Count, typename Weight, typename Need>
__device__ __forceinline__ void find_bin(Shared& S, int n, Count count,
                                         Weight weight, bool by_weight,
                                         uint32_t need_n, Need need_w) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads;
  uint32_t c = 0;
  u64 w = 0;
  for (int i = 0; i < per; ++i) {
    const int bin = tid * per + i;
    if (bin < n) { c += count(bin); w += weight(bin); }
  }
  uint32_t pc = c;
  u64 pw = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t oc = __shfl_up_sync(0xffffffffu, pc, o);
    const u64 ow = __shfl_up_sync(0xffffffffu, pw, o);
    if (lane >= o) { pc += oc; pw += ow; }
  }
  if (lane == 31) { S.warp_n[wid] = pc; S.warp_w[wid] = pw; }
  if (tid == 0) S.found_bin = -1;
  __syncthreads();
  u64 total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const u64 v = S.warp_w[i];
    if (i < wid) { pc += S.warp_n[i]; pw += v; }
    total += v;
  }
  pc -= c;
  pw -= w;
  const u64 need = by_weight ? need_w(total) : 0;
  if (tid == 0) S.target = need;
  for (int i = 0; i < per; ++i) {
    const int bin = tid * per + i;
    if (bin >= n) break;
    const uint32_t nc = pc + count(bin);
    const u64 nw = pw + weight(bin);
    const bool here = by_weight ? pw < need && nw >= need
                                : pc < need_n && nc >= need_n;
    if (here) { S.found_bin = bin; S.found_n = pc; S.found_w = pw; }
    pc = nc;
    pw = nw;
  }
  __syncthreads();
}
// The same of the cluster's bins, as reduce_bins left them.
__device__ void find_bin(Shared& S, int n, bool by_weight, uint32_t need_n,
                         u64 need_w) {
  find_bin(S, n, [&](int i) { return S.all_count[i]; },
           [&](int i) { return S.all_w[i]; }, by_weight, need_n,
           [&](u64) { return need_w; });
}

template <typename T>
__device__ __forceinline__ float logit_at(const T* data, int i) {
  return to_f32(data[i]);
}

// Chunk of the slice that warp `wid` owns in id order: multiples of 128.
__device__ __forceinline__ void warp_chunk(int n, int wid, int* a, int* b) {
  const int per = ((n + kWarps - 1) / kWarps + 127) & ~127;
  *a = min(n, wid * per);
  *b = min(n, *a + per);
}

// Generic selection of the cut by radix on the 64-bit words, most
// significant byte first: the word at which the count reaches need_n (or
// the preceding weight has not yet reached need_w) over the whole cluster.
template <typename T>
__device__ void radix_cut(Shared& S, cg::cluster_group& cl, const T* data,
                          int n, int id0, const Row& r, bool by_weight,
                          uint32_t need_n, u64 need_w) {
  u64 prefix = 0, mask = 0, before_w = 0;
  uint32_t before_n = 0;
  for (int shift = 56; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads)
      S.count[i] = S.w_lo[i] = S.w_hi[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float l = logit_at(data, i);
      if (!(l > -INFINITY)) continue;
      const u64 w = word_of(l, id0 + i);
      if ((w & mask) != prefix) continue;
      const int bin = 255 - (int)(w >> shift & 255);  // larger words first
      atomicAdd(&S.count[bin], 1u);
      add_weight(S, bin, weight_of(x_of(l, r)));
    }
    reduce_bins(S, cl, 256);
    find_bin(S, 256, by_weight, by_weight ? 0 : need_n - before_n,
             by_weight ? need_w - before_w : 0);
    const int bin = S.found_bin;
    before_n += S.found_n;
    before_w += S.found_w;
    prefix |= (u64)(255 - bin) << shift;
    mask |= (u64)255 << shift;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float l = of_key((uint32_t)(prefix >> 32));
    S.cut = prefix;
    S.kept_before = before_w + weight_of(x_of(l, r));
  }
  __syncthreads();
}

// Elements of a 16-byte word.
template <typename T>
struct Vec {
  static constexpr int E = 16 / sizeof(T);
  uint4 w;
  __device__ __forceinline__ float at(int k) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w);
    } else {
      const uint32_t v = k < 2 ? w.x : k < 4 ? w.y : k < 6 ? w.z : w.w;
      return __uint_as_float(k & 1 ? v & 0xffff0000u : v << 16);
    }
  }
};

// f(i, logit) over elements [from, to) of the slice for T threads of index t,
// words of 16 bytes where the data is aligned to them (from always is).
template <typename T, typename F>
__device__ __forceinline__ void each(const T* data, bool wide, int from,
                                     int to, int t, int threads, F f) {
  constexpr int E = Vec<T>::E;
  int done = from;
  if (wide) {
    const int words = (to - from) / E;
    const uint4* p = reinterpret_cast<const uint4*>(data + from);
#pragma unroll 2
    for (int v = t; v < words; v += threads) {
      const Vec<T> x{p[v]};
#pragma unroll
      for (int k = 0; k < E; ++k) f(from + v * E + k, x.at(k));
    }
    done = from + words * E;
  }
  for (int i = done + t; i < to; i += threads) f(i, to_f32(data[i]));
}

// Sorts key[0, n) descending; n at most kCand, entries up to the next power
// of two are overwritten with 0.  Whole CTA.
__device__ void sort_down(u64* key, int n) {
  int P = 2;
  while (P < n) P *= 2;
  for (int i = n + threadIdx.x; i < P; i += kThreads) key[i] = 0;
  __syncthreads();
  for (int k = 2; k <= P; k *= 2) {
    for (int j = k / 2; j > 0; j /= 2) {
      for (int i = threadIdx.x; i < P / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const u64 x = key[a], y = key[b];
        const bool down = (a & k) == 0;
        if ((x < y) == down) {
          key[a] = y;
          key[b] = x;
        }
      }
      // steps within 64 entries stay within a warp's own entries
      if (j > 32 || P / 2 > kThreads) __syncthreads();
      else __syncwarp();
    }
    __syncthreads();
  }
}

// Exclusive sum over the CTA of v (thread order); *all: the total.
__device__ u64 cta_scan(Shared& S, u64 v, u64* all) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  u64 run = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 q = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += q;
  }
  __syncthreads();
  if (lane == 31) S.warp_w[wid] = run;
  __syncthreads();
  u64 before = 0, total = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < wid) before += S.warp_w[i];
    total += S.warp_w[i];
  }
  *all = total;
  return before + run - v;
}

__device__ __forceinline__ u64 draw_target(float u, u64 total) {
  const double f = floor((double)u * (double)total);
  const u64 t = f > 0.0 ? (u64)f : 0;
  return t >= total ? total - 1 : t;
}
__device__ __forceinline__ u64 top_p_bound(float p, u64 total) {
  const double need = ceil((double)p * (double)total);
  return need >= 1.0 ? (u64)need : 1;  // the first token is kept
}

// Gathers S.cand[0, S.listed) of every CTA into S.all_cand of the first, in
// no order; *all: how many, over the cluster.  False, and nothing to use, if
// that is more than kCand.  `call`: a number not used before.  `free`: the
// first CTA's all_cand is not in use.  What it wrote is there after it, and
// nothing of another CTA is read any more.
__device__ bool collect(Shared& S, cg::cluster_group& cl, int call, bool free,
                        int* all) {
  if (free) __syncthreads();
  else cl.sync();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x;
  const uint32_t mine = S.listed;
  if (tid == 0)
    S.list_at = atomicAdd(&cl.map_shared_rank(&S, 0)->row_listed[call], mine);
  if (tid < C) cl.map_shared_rank(&S, tid)->lists[call][rank] = mine;
  __syncthreads();
  const uint32_t at = S.list_at;
  if (at + mine <= kCand) {
    u64* to = cl.map_shared_rank(S.all_cand, 0);
    for (uint32_t i = tid; i < mine; i += kThreads) to[at + i] = S.cand[i];
  }
  cl.sync();
  uint32_t n = 0;
  for (int q = 0; q < C; ++q) n += S.lists[call][q];
  *all = (int)n;
  return n <= kCand;  // the same in every CTA
}

// The cut in the found bin of the histogram: its members gathered in the
// first CTA and sorted, or radix selection if there are too many.  The
// histogram is lost.
template <typename T>
__device__ void bin_cut(Shared& S, cg::cluster_group& cl, const T* data,
                        bool wide, int n, int id0, const Row& r, float t,
                        int call, bool by_weight, uint32_t need_n,
                        u64 need_w) {
  const int tid = threadIdx.x;
  const int bin = S.found_bin;
  const uint32_t before_n = S.found_n;
  const u64 before_w = S.found_w;
  if (tid == 0) S.listed = 0;
  __syncthreads();
  // one comparison on each side decides for most tokens
  const float below = bin_floor(bin, r, t);
  const float above = bin_ceil(bin, r, t);
  each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
    if (l >= below && l <= above && l > -INFINITY && bin_of(l, r) == bin) {
      const uint32_t at = atomicAdd(&S.listed, 1u);
      if (at < kCand) S.cand[at] = word_of(l, id0 + i);
    }
  });
  int all;
  if (!collect(S, cl, call, false, &all)) {
    radix_cut(S, cl, data, n, id0, r, by_weight, need_n, need_w);
    return;
  }
  if (cl.block_rank() == 0) {
    sort_down(S.all_cand, all);
    constexpr int kPer = kCand / kThreads;
    u64 w[kPer], mine = 0, total;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      w[j] = i < all ? weight_of(x_of(of_key((uint32_t)(S.all_cand[i] >> 32)),
                                      r))
                     : 0;
      mine += w[j];
    }
    u64 before = before_w + cta_scan(S, mine, &total);
    const int C = cl.num_blocks();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      const bool last =
          i < all && (by_weight ? before < need_w && before + w[j] >= need_w
                                : before_n + i + 1 == need_n);
      if (last)
        for (int q = 0; q < C; ++q) {
          Shared* o = cl.map_shared_rank(&S, q);
          o->cut = S.all_cand[i];
          o->kept_before = before + w[j];
        }
      before += w[j];
    }
  }
  cl.sync();
}

// The row's n candidates (S.all_cand: its largest tokens, at least k of them)
// to the kept set's cut and size, and the token.  The first k are kept, of
// those the ones whose predecessors weigh less than `bound` (0: p of the k
// tokens' weight).  By sorting them: for ties beyond pick()'s lists.  Whole
// CTA; scratch: S.cand.
__device__ void pick_sorted(Shared& S, const Row& r, int n, int k, u64 bound,
                            float p, float mp, float u, int* token) {
  const int tid = threadIdx.x;
  sort_down(S.all_cand, n);
  constexpr int kPer = kCand / kThreads;
  auto x_at = [&](u64 w) { return x_of(of_key((uint32_t)(w >> 32)), r); };
  float x[kPer];
  u64 w[kPer], mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    x[j] = i < k ? x_at(S.all_cand[i]) : 0.f;
    w[j] = i < k ? weight_of(x[j]) : 0;
    mine += w[j];
  }
  u64 total, before = cta_scan(S, mine, &total);
  if (bound == 0) bound = p < 1.f ? top_p_bound(p, total) : ~0ull;
  int kept = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    if (i < k && (i == 0 || before < bound) && x[j] >= mp) ++kept;
    before += w[j];
  }
  u64 all;
  cta_scan(S, (u64)kept, &all);
  kept = (int)all;  // a prefix of the order
  if (tid == 0) {
    S.cut = S.all_cand[kept - 1];
    S.kept = kept;
  }
  // the kept tokens by id: the word's lower half is the id's complement
  for (int i = tid; i < kept; i += kThreads)
    S.cand[i] = S.all_cand[i] << 32 | (uint32_t)i;
  __syncthreads();
  sort_down(S.cand, kept);
  mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    w[j] = i < kept ? weight_of(x_at(S.all_cand[(uint32_t)S.cand[i]])) : 0;
    mine += w[j];
  }
  before = cta_scan(S, mine, &total);
  const u64 target = draw_target(u, total);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = tid * kPer + j;
    if (w[j] > 0 && target >= before && target < before + w[j])
      *token = (int)~(uint32_t)(S.cand[i] >> 32);
    before += w[j];
  }
}

// The same without a sort.  Bins of equal width from the maximum to `low`
// (which no candidate is below) hold the candidates' numbers and weights: the
// bin of the k-th token, or of the one whose weight passes the bound, is found
// by a scan, and its few members by comparing each with each.  The token is
// found likewise, in bins of ids.  1053 candidates, k = 1000, p = 0.9: sorting
// them by rank, then those kept by id, took 33 us of a lone row's 41 us.
__device__ void pick(Shared& S, const Row& r, float t, float low, int V, int n,
                     int k, u64 bound, float p, float mp, float u,
                     int* token) {
  const int tid = threadIdx.x;
  const u64 given = bound;
  const float span = low > -INFINITY ? r.top - low : 32.f * t;
  const float scale = (float)(kBins - 1) / span;
  int shift = 0;
  while (V - 1 >> shift >= kBins) ++shift;
  auto clear = [&] {
    for (int i = tid; i < kBins; i += kThreads)
      S.count[i] = S.w_lo[i] = S.w_hi[i] = 0;
    if (tid == 0) S.n_list = 0;
    __syncthreads();
  };
  auto logit = [&](u64 w) { return of_key((uint32_t)(w >> 32)); };
  auto bin_at = [&](u64 w) {  // monotone; what is no number counts as 0
    return min((int)__fmul_rn(__fsub_rn(r.top, logit(w)), scale), kBins - 1);
  };
  auto id_bin = [&](u64 w) { return (int)(~(uint32_t)w >> shift); };
  auto count = [&](int i) { return S.count[i]; };
  auto weight = [&](int i) { return (u64)S.w_hi[i] << 32 | S.w_lo[i]; };
  auto list = [&](u64 key, float x) {
    const uint32_t at = atomicAdd(&S.n_list, 1u);
    if (at < kList) {
      S.list[at] = key;
      S.list_w[at] = weight_of(x);
    }
  };
  // The cut in the found bin; false if it has too many members.
  auto edge = [&](bool by_weight) {
    const int bin = S.found_bin;
    for (int i = tid; i < n; i += kThreads) {
      const u64 c = S.all_cand[i];
      if (bin_at(c) == bin) list(c, x_of(logit(c), r));
    }
    __syncthreads();
    const int m = (int)S.n_list;
    if (m > kList) return false;
    if (tid < m) {
      const u64 mine = S.list[tid], w = S.list_w[tid], need = S.target;
      int rank = (int)S.found_n;
      u64 before = S.found_w;
      for (int j = 0; j < m; ++j)
        if (S.list[j] > mine) {
          ++rank;
          before += S.list_w[j];
        }
      if (by_weight ? before < need && before + w >= need : rank + 1 == k) {
        S.cut = mine;
        S.kept_before = before + w;
      }
    }
    __syncthreads();
    if (tid == 0) S.n_list = 0;
    return true;
  };

  if (tid == 0) {
    S.kept = 0;
    S.least_key = ~0u;
  }
  clear();
  for (int i = tid; i < n; i += kThreads) {
    const u64 c = S.all_cand[i];
    const int b = bin_at(c);
    atomicAdd(&S.count[b], 1u);
    add_weight(S, b, weight_of(x_of(logit(c), r)));
  }
  __syncthreads();
  bool found = false, ok = true;
  if (bound) {
    find_bin(S, kBins, count, weight, true, 0, [&](u64) { return bound; });
    found = S.found_bin >= 0;
    if (found) ok = edge(true);
    else __syncthreads();  // all of them are lighter: all are kept
  }
  if (!found) {
    find_bin(S, kBins, count, weight, false, (uint32_t)k,
             [](u64) { return 0ull; });
    ok = edge(false);
    if (ok && bound == 0 && p < 1.f) {
      bound = top_p_bound(p, S.kept_before);
      find_bin(S, kBins, count, weight, true, 0, [&](u64) { return bound; });
      ok = edge(true);
    }
  }
  if (ok) {
    const u64 cut = S.cut;
    auto keeps = [&](u64 c, float x) { return c >= cut && x >= mp; };
    clear();
    for (int i = tid; i < n; i += kThreads) {
      const u64 c = S.all_cand[i];
      const float x = x_of(logit(c), r);
      if (!keeps(c, x)) continue;
      add_weight(S, id_bin(c), weight_of(x));
      atomicAdd(&S.kept, 1);
      if (mp > 0.f) atomicMin(&S.least_key, (uint32_t)(c >> 32));
    }
    __syncthreads();
    find_bin(S, kBins, count, weight, true, 0,
             [&](u64 total) { return draw_target(u, total) + 1; });
    const int bin = S.found_bin;
    for (int i = tid; i < n; i += kThreads) {
      const u64 c = S.all_cand[i];
      if (id_bin(c) != bin) continue;
      const float x = x_of(logit(c), r);
      if (keeps(c, x)) list(~(uint32_t)c, x);
    }
    // what is kept, as one cut: all of the smallest logit if min-p decided
    if (tid == 0 && mp > 0.f)
      S.cut = max(cut, (u64)S.least_key << 32 | 0x80000000u);
    __syncthreads();
    const int m = (int)S.n_list;
    ok = m <= kList;
    if (ok && tid < m) {
      const u64 mine = S.list[tid], target = S.target - 1;
      u64 before = S.found_w;
      for (int j = 0; j < m; ++j)
        if (S.list[j] < mine) before += S.list_w[j];
      if (target >= before && target < before + S.list_w[tid])
        *token = (int)mine;
    }
  }
  if (!ok) pick_sorted(S, r, n, k, given, p, mp, u, token);
}

// Three CTAs to an SM (40 registers) hide each other's barriers: 288 rows with
// mixed filters 217 us with two (64 registers), 193 us with three, 191 us with
// four, where 128 rows without filters go from 73 us to 78 us.
template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
    sample_kernel(const __grid_constant__ SampleArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ uint4 smem16[];
  Shared& S = *reinterpret_cast<Shared*>(smem16);
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / C;
  const int id0 = rank * a.slice;
  const int n = max(0, min(a.slice, a.V - id0));
  const T* src = static_cast<const T*>(a.logits) + row * a.ld + id0;
  T* own = reinterpret_cast<T*>(smem16 + (sizeof(Shared) + 15) / 16);
  const T* data = a.resident ? own : src;
  const bool src_wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  const bool wide = a.resident || src_wide;

  // ---- the slice and the row's maximum -------------------------------------
  if (tid == 0) {
    S.odd = 0;
    S.kept_n = 0;
    S.listed = 0;
    for (int i = 0; i < kCollects; ++i) S.row_listed[i] = 0;
    S.first = 0x7fffffff;
    S.t = a.temperature[row];
    S.top_k = a.top_k ? a.top_k[row] : 0;
    S.top_p = a.top_p ? a.top_p[row] : 1.f;
    S.min_p = a.min_p ? a.min_p[row] : 0.f;
    S.u = a.u[row];
    for (int i = 0; i < kChunks; ++i) tc::mbar_init(&S.landed[i], 1);
    tc::fence_mbar_init();
  }
  __syncthreads();
  float tops[kChunks];  // of this thread's tokens, by quarters
#pragma unroll
  for (int c = 0; c < kChunks; ++c) tops[c] = -INFINITY;
  bool odd = false;  // a logit that is not finite
  auto take = [&](int c, float l) {
    odd |= !(fabsf(l) < INFINITY);
    tops[c] = fmaxf(tops[c], l);    // passes over a NaN
  };
  // A word of them; bf16 in pairs: what is not finite survives one of the
  // largest of the pairs and the smallest.
  auto take_word = [&](int c, const Vec<T>& x) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int k = 0; k < Vec<T>::E; ++k) take(c, x.at(k));
    } else {
      const __nv_bfloat162* v =
          reinterpret_cast<const __nv_bfloat162*>(&x.w);
      const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(v[0], v[1]),
                                            __hmax2_nan(v[2], v[3]));
      const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(v[0], v[1]),
                                            __hmin2_nan(v[2], v[3]));
      const float2 h = __bfloat1622float2(hi), l = __bfloat1622float2(lo);
      if (fabsf(h.x) < INFINITY && fabsf(h.y) < INFINITY &&
          l.x > -INFINITY && l.y > -INFINITY) {
        tops[c] = fmaxf(tops[c], fmaxf(h.x, h.y));
      } else {
#pragma unroll
        for (int k = 0; k < Vec<T>::E; ++k) take(c, x.at(k));
      }
    }
  };
  if (src_wide && a.resident) {
    constexpr int E = Vec<T>::E;
    const int words = n / E, per = (words + kChunks - 1) / kChunks;
    if (tid == 0)
      for (int c = 0; c < kChunks; ++c) {
        const int v0 = min(words, c * per), v1 = min(words, v0 + per);
        tc::mbar_arrive_expect_tx(&S.landed[c], (v1 - v0) * 16);
        if (v1 > v0)
          tc::bulk_load(reinterpret_cast<uint4*>(own) + v0,
                        reinterpret_cast<const uint4*>(src) + v0,
                        (v1 - v0) * 16, &S.landed[c]);
      }
    int give_up = 0;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (!tc::mbar_wait_bounded(&S.landed[c], 0, &give_up, kWait))
        raise_error(a.err, kErrTimeout);
      const int v1 = min(words, (c + 1) * per);
#pragma unroll 4
      for (int v = min(words, c * per) + tid; v < v1; v += kThreads) {
        const Vec<T> x{reinterpret_cast<const uint4*>(own)[v]};
        take_word(c, x);
      }
    }
    for (int i = words * E + tid; i < n; i += kThreads) {
      const T x = src[i];
      own[i] = x;
      take(0, to_f32(x));
    }
  } else if (src_wide) {
    constexpr int E = Vec<T>::E;
    const int words = n / E;
    const uint4* p = reinterpret_cast<const uint4*>(src);
    for (int v = tid; v < words; v += kChunks * kThreads) {
      Vec<T> x[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (v + c * kThreads < words) x[c].w = p[v + c * kThreads];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (v + c * kThreads < words) take_word(c, x[c]);
    }
    for (int i = words * E + tid; i < n; i += kThreads)
      take(0, to_f32(src[i]));
  } else {
    for (int i0 = tid; i0 < n; i0 += kChunks * kThreads) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int i = i0 + c * kThreads;
        if (i < n) {
          const T x = src[i];
          if (a.resident) own[i] = x;
          take(c, to_f32(x));
        }
      }
    }
  }
  float top = tops[0];
#pragma unroll
  for (int c = 1; c < kChunks; ++c) top = fmaxf(top, tops[c]);
  top = warp_max(top);
  if (lane == 0) S.warp_w[wid] = __float_as_uint(top);
  __syncthreads();
  if (odd) S.odd = 1;
  if (tid == 0) {
    for (int i = 1; i < kWarps; ++i)
      top = fmaxf(top, __uint_as_float((uint32_t)S.warp_w[i]));
    S.top = top;
  }
  cl.sync();
  top = lane < C ? cl.map_shared_rank(&S, lane)->top : -INFINITY;
  top = warp_max(top);

  Row r;
  const float t = S.t;
  r.top = top;
  r.greedy = !(t > 0.f && t < INFINITY);
  r.inv_t = r.greedy ? 0.f : __fdiv_rn(1.f, t);
  const bool empty = top == -INFINITY;
  if (tid == 0 && (empty || !(t >= 0.f && t < INFINITY)))
    raise_error(a.err, kErrNonfinite);
  if (S.odd) {  // -inf is a masked token, the others are errors
    bool bad = false;
    each(data, wide, 0, n, tid, kThreads,
         [&](int, float l) { bad |= !(l < INFINITY); });
    if (bad) raise_error(a.err, kErrNonfinite);
  }
  const int k = S.top_k;
  const float p = S.top_p;
  // at most 1 (which keeps the maximum), 0 for what is no number
  const float mp = S.min_p > 0.f ? fminf(S.min_p, 1.f) : 0.f;
  const float u = S.u;
  const bool by_k = !r.greedy && !empty && k > 0 && k < a.V;
  const bool by_p = !r.greedy && !empty && p < 1.f;
  float* dst = a.filtered ? a.filtered + (size_t)row * a.V + id0 : nullptr;
  // the slice's filtered logits: those not below the cut, given as a word
  auto filter = [&](u64 cut) {
    const float lc = of_key((uint32_t)(cut >> 32));
    const int last = (int)~(uint32_t)cut;  // of the tokens with that logit
    if (wide && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
      const int words = n / 4;
#pragma unroll 2
      for (int v = tid; v < words; v += kThreads) {
        float f[4];
        if constexpr (sizeof(T) == 4) {
          const float4 x = reinterpret_cast<const float4*>(data)[v];
          f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        } else {
          const uint2 x = reinterpret_cast<const uint2*>(data)[v];
          f[0] = __uint_as_float(x.x << 16);
          f[1] = __uint_as_float(x.x & 0xffff0000u);
          f[2] = __uint_as_float(x.y << 16);
          f[3] = __uint_as_float(x.y & 0xffff0000u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[j] = f[j] > lc || (f[j] == lc && id0 + 4 * v + j <= last)
                     ? f[j] : -INFINITY;
        reinterpret_cast<float4*>(dst)[v] =
            make_float4(f[0], f[1], f[2], f[3]);
      }
      for (int i = words * 4 + tid; i < n; i += kThreads) {
        const float l = to_f32(data[i]);
        dst[i] = l > lc || (l == lc && id0 + i <= last) ? l : -INFINITY;
      }
    } else {
      for (int i = tid; i < n; i += kThreads) {
        const float l = to_f32(data[i]);
        dst[i] = l > lc || (l == lc && id0 + i <= last) ? l : -INFINITY;
      }
    }
  };

  // ---- T = 0, or nothing to draw from --------------------------------------
  if (r.greedy || empty) {  // uniform over the cluster
    int first = 0x7fffffff;
    if (!empty)
      each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
        if (l == top) first = min(first, id0 + i);
      });
    if (first != 0x7fffffff) atomicMin(&S.first, first);
    cl.sync();
    first = lane < C ? cl.map_shared_rank(&S, lane)->first : 0x7fffffff;
#pragma unroll
    for (int o = 16; o; o >>= 1)
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
    if (rank == 0 && tid == 0) {
      a.token[row] = empty ? -1 : first;
      if (a.n_kept) a.n_kept[row] = empty ? 0 : 1;
    }
    if (dst) filter(empty ? ~0ull : word_of(top, first));
    cl.sync();  // no CTA leaves while another reads its maximum
    return;
  }

  // The tokens from `low` up as candidates, cut and drawn from by the first
  // CTA; false if they are too many.
  auto finish = [&](float low, bool free, int most, u64 bound) {
    each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
      if (l >= low && l > -INFINITY) {
        const uint32_t at = atomicAdd(&S.listed, 1u);
        if (at < kCand) S.cand[at] = word_of(l, id0 + i);
      }
    });
    int all;
    if (!collect(S, cl, 0, free, &all)) return false;
    if (rank == 0) {
      pick(S, r, t, low, a.V, all, min(most, all), bound, p, mp, u,
           a.token + row);
      if (tid == 0 && a.n_kept) a.n_kept[row] = S.kept;
      __syncthreads();
      if (dst && tid < C) cl.map_shared_rank(&S, tid)->cut = S.cut;
    }
    if (dst) {
      cl.sync();
      filter(S.cut);
    }
    return true;  // nothing of another CTA is read any more
  };

  // ---- top-k: candidates from the threads' maxima -----------------------------
  if (by_k && k <= kCand) {
    // bins of the threads' maxima, half as fine as the weights' bins; below
    // the slice's own maximum where each CTA takes its own bound
    const bool own_bound = k <= kOwnBound;
    Row b = r;
    if (own_bound) b.top = S.top;
    for (int i = tid; i < kCandBins; i += kThreads) S.count[i] = 0;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (tops[c] > -INFINITY)
        atomicAdd(&S.count[bin_of(tops[c], b) / (kBins / kCandBins)], 1u);
    if (own_bound) {
      __syncthreads();
    } else {
      cl.sync();
      for (int i = tid; i < kCandBins; i += kThreads) {
        uint32_t c = 0;
        for (int q = 0; q < C; ++q) c += cl.map_shared_rank(&S, q)->count[i];
        S.all_count[i] = c;
      }
      __syncthreads();
    }
    const uint32_t* of = own_bound ? S.count : S.all_count;
    find_bin(S, kCandBins, [&](int i) { return of[i]; },
             [](int) { return 0ull; }, false, (uint32_t)k,
             [](u64) { return 0ull; });
    const int bin = S.found_bin;
    // the counts have been read; the lists take their place
    if (own_bound) __syncthreads();
    else cl.sync();
    const float low =
        bin < 0 ? -INFINITY
                : bin_floor((bin + 1) * (kBins / kCandBins) - 1, b, t);
    // top-k of fewer tokens than k keeps them all
    if (finish(low, true, k, 0)) return;
  }

  // ---- the cut by histogram of weights --------------------------------------
  u64 cut = 0;
  if (by_k || by_p) {
    for (int i = tid; i < kBins; i += kThreads)
      S.count[i] = S.w_lo[i] = S.w_hi[i] = 0;
    __syncthreads();
    // Top-p only: tokens of less than (1 - p) W / V weigh less than (1 - p) W
    // together, so they are past the cut and need no bin.  The weight of this
    // CTA's threads' maxima, times 0.9 for roundings, stands for W from below.
    float low = -INFINITY;
    if (!by_k) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (tops[c] > -INFINITY) sum += x_of(tops[c], r);
      sum = warp_sum(sum);
      if (lane == 0) S.warp_n[wid] = __float_as_uint(sum);
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < kWarps; ++i) sum += __uint_as_float(S.warp_n[i]);
      __syncthreads();
      const float least = 0.9f * (1.f - p) * sum / (float)a.V;
      if (least > 0.f && least < 1.f)
        low = r.top + logf(least) * t * 1.0001f - fabsf(r.top) * 1e-6f;
    }
    const bool plain = !S.odd && r.inv_t < INFINITY;
    auto fill = [&] {
      u64 sum = 0;
      if (plain) {  // as in the sum of all weights below
        for (int b = 0; b < n; b += kThreads * 512) {
          uint32_t hi = 0, lo = 0, m = 0;
          each(data, wide, b, min(n, b + kThreads * 512), tid, kThreads,
               [&](int, float l) {
                 const WeightBits w = weight_bits(x_plain(l, r));
                 hi += w.hi;
                 lo += w.lo;
                 ++m;
                 if (l < low) return;
                 const int bin = bin_of(l, r);
                 atomicAdd(&S.count[bin], 1u);
                 if (by_p)
                   add_weight(S, bin,
                              (u64)(w.hi - 0x4b000000u) * (1u << 23) +
                                  (w.lo - 0x4b000000u));
               });
          sum += (u64)(hi - m * 0x4b000000u) * (1u << 23) +
                 (lo - m * 0x4b000000u);
        }
        return sum;
      }
      each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
        if (!(l > -INFINITY)) return;
        const u64 w = weight_of(x_of(l, r));
        sum += w;
        if (l < low) return;
        const int bin = bin_of(l, r);
        atomicAdd(&S.count[bin], 1u);
        if (by_p) add_weight(S, bin, w);
      });
      return sum;
    };
    bool redo = false;  // the top-k cut has overwritten the histogram
    u64 sum = warp_total(fill());
    if (lane == 0) S.warp_w[wid] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < kWarps; ++i) sum += S.warp_w[i];
      S.total = sum;
    }
    reduce_bins(S, cl, kBins);
    u64 total = 0;
    for (int c = 0; c < C; ++c) total += cl.map_shared_rank(&S, c)->total;
    if (by_k) {
      find_bin(S, kBins, false, (uint32_t)k, 0);
      if (S.found_bin >= 0) {  // fewer than k tokens above -inf: no cut
        redo = true;
        bin_cut(S, cl, data, wide, n, id0, r, t, 1, false, (uint32_t)k, 0);
        cut = S.cut;
        total = S.kept_before;
        __syncthreads();
      }
    }
    if (by_p) {
      const u64 bound = top_p_bound(p, total);
      // The tokens past the top-k cut may stay in the histogram: bound is at
      // most the weight before them.
      if (redo) {
        for (int i = tid; i < kBins; i += kThreads)
          S.count[i] = S.w_lo[i] = S.w_hi[i] = 0;
        __syncthreads();
        fill();
        reduce_bins(S, cl, kBins);
      }
      find_bin(S, kBins, true, 0, bound);
      // few tokens up to the cut's bin: they are all that is left to look at
      const int bin = S.found_bin;
      if (!redo && bin < kBins - 1 &&
          S.found_n + S.all_count[bin] <= kCand / 2) {
        if (tid == 0) S.listed = 0;
        __syncthreads();
        if (finish(bin_floor(bin, r, t), false, kCand, bound)) return;
        // (not so few: the bins have been overwritten)
        for (int i = tid; i < kBins; i += kThreads)
          S.count[i] = S.w_lo[i] = S.w_hi[i] = 0;
        __syncthreads();
        fill();
        reduce_bins(S, cl, kBins);
        find_bin(S, kBins, true, 0, bound);
      }
      bin_cut(S, cl, data, wide, n, id0, r, t, 2, true, 0, bound);
      cut = max(cut, S.cut);
    }
  }
  const bool by_m = mp > 0.f;
  auto keeps = [&](float l, int i, float x) {
    return l > -INFINITY && (cut == 0 || word_of(l, id0 + i) >= cut) &&
           (!by_m || x >= mp);
  };

  // ---- kept weights in id order, the draw, the filtered logits -------------
  int c0, c1;
  warp_chunk(n, wid, &c0, &c1);
  u64 sum = 0;
  uint32_t cnt = 0;
  float least = INFINITY;  // smallest kept logit, where min-p has a say
  if (cut == 0 && !by_m) {
    if (S.odd || !(r.inv_t < INFINITY)) {  // uniform in the CTA
      each(data, wide, c0, c1, lane, 32, [&](int, float l) {
        const bool on = l > -INFINITY;  // not a NaN, either
        sum += weight_of(on ? x_of(l, r) : 0.f);
        cnt += on;
      });
    } else {
      // All weights are wanted and all logits finite.  The halves of up to
      // 512 weights fit 32 bits each; the 0x4b000000 of every float comes
      // off at the end.
      for (int b = c0; b < c1; b += 32 * 512) {
        const int e = min(c1, b + 32 * 512);
        uint32_t hi = 0, lo = 0, m = 0;
        each(data, wide, b, e, lane, 32, [&](int, float l) {
          const WeightBits w = weight_bits(x_plain(l, r));
          hi += w.hi;
          lo += w.lo;
          ++m;
        });
        sum += (u64)(hi - m * 0x4b000000u) * (1u << 23) +
               (lo - m * 0x4b000000u);
        cnt += m;
      }
    }
  } else {
    // no weight is needed of what lies surely below the filters
    const float low =
        fmaxf(cut ? of_key((uint32_t)(cut >> 32)) : -INFINITY,
              by_m ? r.top + logf(mp) * t * 1.0001f - fabsf(r.top) * 1e-6f
                   : -INFINITY);
    each(data, wide, c0, c1, lane, 32, [&](int i, float l) {
      if (!(l >= low)) return;
      const float x = x_of(l, r);
      if (keeps(l, i, x)) {
        sum += weight_of(x);
        ++cnt;
        least = fminf(least, l);
      }
    });
  }
  least = -warp_max(-least);
  sum = warp_total(sum);
  cnt = warp_total(cnt);
  if (lane == 0) {
    S.kept_w[wid] = sum;
    S.kept_least[wid] = least;
    if (cnt) atomicAdd(&S.kept_n, cnt);
  }
  cl.sync();
  if (dst) {
    // what is kept, as one cut: all tokens of the smallest kept logit if
    // min-p decided, all above -inf if nothing did
    u64 at = cut ? cut : (u64)kKeyNegInf << 32;
    if (by_m) {
      least = INFINITY;
      for (int i = lane; i < C * kWarps; i += 32)
        least = fminf(least, cl.map_shared_rank(&S, i / kWarps)
                                 ->kept_least[i % kWarps]);
      least = -warp_max(-least);
      at = max(at, word_of(least, 0x7fffffff));  // up to the last id
    }
    filter(at);
  }
  if (wid == 0) {
    // kept weight of every (CTA, warp) chunk in id order: lane handles four
    constexpr int kPer = kMaxCluster * kWarps / 32;
    u64 w[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = lane * kPer + j;
      w[j] = at < C * kWarps
                 ? cl.map_shared_rank(&S, at / kWarps)->kept_w[at % kWarps]
                 : 0;
      mine += w[j];
    }
    u64 run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    const u64 total = __shfl_sync(0xffffffffu, run, 31);
    if (rank == 0) {
      uint32_t nk = lane < C ? cl.map_shared_rank(&S, lane)->kept_n : 0;
      nk = warp_total(nk);
      if (lane == 0 && a.n_kept) a.n_kept[row] = (int)nk;
    }
    const u64 target = draw_target(u, total);
    u64 before = run - mine;
    int hit = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (hit < 0 && target >= before && target < before + w[j])
        hit = lane * kPer + j;
      if (hit < 0) before += w[j];
    }
    const unsigned who = __ballot_sync(0xffffffffu, hit >= 0);
    const int from = __ffs(who) - 1;
    hit = __shfl_sync(0xffffffffu, hit, from);
    before = __shfl_sync(0xffffffffu, before, from);
    if (hit / kWarps == rank) {  // the chunk is in this CTA's slice
      warp_chunk(n, hit % kWarps, &c0, &c1);
      // eight tokens to a lane at a time
      for (int base = c0; base < c1; base += 256) {
        u64 v[8], one = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = base + lane * 8 + j;
          const float l = i < c1 ? to_f32(data[i]) : -INFINITY;
          const float x = x_of(l, r);
          v[j] = i < c1 && keeps(l, i, x) ? weight_of(x) : 0;
          one += v[j];
        }
        u64 sum8 = one;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 q = __shfl_up_sync(0xffffffffu, sum8, o);
          if (lane >= o) sum8 += q;
        }
        u64 at = before + sum8 - one;
        const bool here = one > 0 && target >= at && target < at + one;
        if (here) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (target >= at && target < at + v[j])
              a.token[row] = id0 + base + lane * 8 + j;
            at += v[j];
          }
        }
        if (__any_sync(0xffffffffu, here)) break;
        before += __shfl_sync(0xffffffffu, sum8, 31);
      }
    }
  }
  cl.sync();  // no CTA leaves while another reads its sums
}

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  // Up to eight CTAs for each SM, three of them resident, if that takes at
  // most eight to a row.  Fewer to a row cost less in barriers between them,
  // more of them shorten rows that need several passes (288 rows of 151936
  // fp32 logits with mixed filters: 235 us with two, 193 us with four; a lone
  // row of top-k 50: 28 us with two, 20 us with eight; against that 128 rows
  // of 262144 without filters: 68 us with four, 73 us with eight).  Never
  // more than slices of 4096 tokens need.
  int C = kMaxCluster;
  while (C > 1 && ((long long)a.R * C > 8 * 152 ||
                   (long long)(C / 2) * 4096 >= a.V))
    C /= 2;
  // A slice stays in shared memory where two CTAs fit an SM so; the rest is
  // read again, from L2 for the most part.
  a.slice = (int)((((long long)a.V + C - 1) / C + 7) & ~7ll);
  a.resident = (long long)a.slice * (long long)sizeof(T) <= 76 * 1024;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 +
                      (a.resident ? (size_t)a.slice * sizeof(T) : 16);
  auto* f = sample_kernel<T>;
  cudaError_t e = cudaFuncSetAttribute(
      f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3((unsigned)a.R * C), dim3(kThreads), smem, s, C);
  return cudaLaunchKernelEx(&L.cfg, f, a);
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_sample_workspace_bytes(int R, int V) {
  if (R < 1 || R > (1 << 24) || V < 1 || V > (1 << 30)) return 0;
  return 256;
}

dflash_status dflash_sample(const void* logits, int64_t ld, dflash_dtype dt,
                            const float* temperature, const int32_t* top_k,
                            const float* top_p, const float* min_p,
                            const float* u, int R, int V, int32_t* token,
                            int32_t* n_kept, float* filtered, void* ws,
                            size_t ws_bytes, dflash_stream_t stream) {
  using namespace dflash;
  if (!(logits && temperature && u && token && ws))
    return DFLASH_ERR_INVALID_ARG;
  if (dt != DFLASH_BF16 && dt != DFLASH_FP32) return DFLASH_ERR_INVALID_ARG;
  const size_t need = dflash_sample_workspace_bytes(R, V);
  if (need == 0 || ws_bytes < need || ld < V) return DFLASH_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  SampleArgs a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.logits = logits;
  a.ld = ld;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.R = R;
  a.V = V;
  a.token = token;
  a.n_kept = n_kept;
  a.filtered = filtered;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == DFLASH_FP32 ? launch<float>(a, s)
                                          : launch<__nv_bfloat16>(a, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
