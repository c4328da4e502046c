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
// A cluster of CTAs owns a row: each CTA reads its slice from HBM once, and
// later passes from L2, or from shared memory where few CTAs leave room for
// the slice (by bulk copies: more bytes in flight than its threads could
// have); only maxima, histograms, short lists and sums travel between the CTAs
// (distributed shared memory).
// What happens then is the row's own:
//   T = 0           the first maximum;
//   top-k           the k-th largest of the threads' own maxima bounds the
//                   k-th largest token from below, and only the threads'
//                   parts whose maximum reaches it are read again for the few
//                   more than k candidates (with small k each CTA takes its
//                   own bound, which spares two cluster barriers); one CTA
//                   finds the cut in them, with top-p and min-p, and draws
//                   among them;
//   min-p only      likewise from its bound, if the tokens are few;
//   top-p only      the weights' sum, and the tokens' numbers in bins of
//                   (max - l) / T, from which any prefix's weight is known to
//                   a part in 64: a short prefix is gathered and cut as above;
//                   of a long one the weight before a range of bins around the
//                   cut is summed and the range's members gathered and cut;
//   neither         kept weights by warp chunk, the draw.
// What overflows a list (ties by the thousand, a tail of weightless tokens)
// is resolved by a histogram of the 64-bit words instead, refined until the
// rest fits one.
//
// What bounds it.  288 rows of 151936 fp32 logits, 26 us of HBM: T = 0 44 us,
// top-k 50 61 us, no filter 77 us, top-k 1000 with top-p 87 us, min-p 0.001
// (6600 tokens) 153 us, top-p 0.9 (16600 tokens) 195 us: the loads' latency
// (the second reading from L2 among them) and the barriers of each row's chain,
// which other rows' CTAs hide in part (issue slots are used to 30 to 55 %).  A
// lone row that L2 holds: 8, 13, 10, 19, 16 and 30 us, the chain alone.
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
constexpr int kBins = 2048;
constexpr float kBinsPerUnit = 64.f;   // bins of 1/64 in (max - l) / T
constexpr int kTopBins = 192;          // bins whose weight is summed
constexpr int kSlots = 1024;           // bins of candidates
constexpr int kCand = 2048;            // candidates, over the cluster
constexpr int kOwn = 1536;             // of one CTA
constexpr int kOwnBound = 128;         // largest k for a bound of each CTA
constexpr int kChunks = 4;             // copies of a slice
// Weights whose halves a thread adds up in 32 bits: 512 halves of 23 bits fit.
// In a block of this many tokens to a thread, each() gives it one more where
// the last word is not full.
constexpr int kBlock = 504;            // (words of eight)
constexpr int kCandBins = 512;         // bins of 1/16 for a bound of them
constexpr int kList = 256;             // members of one bin
constexpr int kCollects = 5;           // lists that a row may gather
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
  uint64_t wait_ns;  // limit of the waits for the slice's copies
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
  float top;             // largest logit of the slice; NaN: it did not come
  int first;             // T = 0: first token of the slice that has it
  u64 total;             // weight of the slice
  u64 top_w;             // and of its tokens in the first kTopBins bins
  u64 kept_w[kWarps];    // kept weight of each warp's chunk
  float kept_least[kWarps];  // and its smallest kept logit
  uint32_t kept_n;
  uint32_t odd;          // a logit of the slice is not finite
  uint32_t fine;         // one has more bits than bf16
  uint32_t lists[kCollects][kMaxCluster];  // lengths of every CTA's lists
  uint32_t row_listed[kCollects];  // the first CTA's: places taken in all_cand
  uint64_t landed[kChunks];  // barriers of the slice's copies
  // this CTA's own
  uint32_t listed, n_quarters;
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
  uint32_t late;         // a copy of the slice did not come in time
  // (at 8 bytes beside a multiple of 16 a lone row took 11.5 us, not 11.1)
  union alignas(16) {
    struct {
      union {
        uint32_t count[kBins];  // read by the cluster
        struct {
          uint32_t slots[kSlots];
          u64 list[kList], list_w[kList];
        };
      };
      union {
        struct {
          uint32_t w_lo[kSlots], w_hi[kSlots];  // read by the cluster
        };
        uint32_t all_count[kBins];
      };
      uint32_t all_n[kSlots];
      u64 all_w[kSlots];
    };
    struct {
      u64 cand[kOwn];       // this CTA's candidates
      uint16_t quarters[kChunks * kThreads];  // that may have some
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

// The three bounds below are differences from the maximum.  Under an infinite
// one there are its own tokens, in bin 0, and all others, weightless and in the
// last bin; the bounds are then these tokens' own logits.

// A logit below all of bins 0 .. bin (-inf after the last): z is less than
// (bin + 1) / kBinsPerUnit there, with room for its roundings.
__device__ __forceinline__ float bin_floor(int bin, const Row& r, float t) {
  if (bin >= kBins - 1) return -INFINITY;
  if (r.top == INFINITY) return r.top;
  const float z = (float)(bin + 1) / kBinsPerUnit;
  return r.top - z * t * 1.0001f - fabsf(r.top) * 1e-6f;
}

// A logit above all of bins bin, bin + 1, ...
__device__ __forceinline__ float bin_ceil(int bin, const Row& r, float t) {
  if (r.top == INFINITY) return bin > 0 ? 0x1.fffffep127f : r.top;
  const float z = (float)bin / kBinsPerUnit;
  return r.top - z * t * 0.9999f + fabsf(r.top) * 1e-6f;
}

// A logit below all that weigh x or more (0 < x <= 1).
__device__ __forceinline__ float weight_floor(float x, const Row& r, float t) {
  if (r.top == INFINITY) return r.top;
  return r.top + logf(x) * t * 1.0001f - fabsf(r.top) * 1e-6f;
}

__device__ __forceinline__ void add_weight(Shared& S, int bin, u64 w) {
  const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
  const uint32_t old = atomicAdd(&S.w_lo[bin], lo);
  const uint32_t up = hi + (old + lo < old ? 1u : 0u);
  if (up) atomicAdd(&S.w_hi[bin], up);
}

// Sums the cluster's counts (first n bins) into all_count of every CTA.
// Cluster barriers on both sides: the counts are complete before, and may be
// overwritten after.
__device__ void reduce_counts(Shared& S, cg::cluster_group& cl, int n) {
  cl.sync();
  const int C = cl.num_blocks();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint32_t c = 0;
    for (int q = 0; q < C; ++q) c += cl.map_shared_rank(&S, q)->count[i];
    S.all_count[i] = c;
  }
  cl.sync();
}

// The first of n bins (N at most) at which the running count reaches `need_n`
// (by_weight false) or the running weight reaches need_w(weight of all bins);
// its predecessors' sums.  found_bin = -1 if none does.  Whole CTA, which has
// left the last call's results behind.
template <int N, typename Count, typename Weight, typename Need>
__device__ __forceinline__ void find_bin(Shared& S, int n, Count count,
                                         Weight weight, bool by_weight,
                                         uint32_t need_n, Need need_w) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  constexpr int kPer = (N + kThreads - 1) / kThreads;
  uint32_t c[kPer], pc = 0;
  u64 w[kPer], pw = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int bin = tid * kPer + i;
    c[i] = bin < n ? count(bin) : 0;
    w[i] = bin < n ? weight(bin) : 0;
    pc += c[i];
    pw += w[i];
  }
  const uint32_t own_c = pc;
  const u64 own_w = pw;
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
  pc -= own_c;
  pw -= own_w;
  const u64 need = by_weight ? need_w(total) : 0;
  if (tid == 0) S.target = need;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool here = by_weight ? pw < need && pw + w[i] >= need
                                : pc < need_n && pc + c[i] >= need_n;
    if (here) {
      S.found_bin = tid * kPer + i;
      S.found_n = pc;
      S.found_w = pw;
    }
    pc += c[i];
    pw += w[i];
  }
  __syncthreads();
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
// Not unrolled: other warps hide the loads, and registers are short.
template <typename T, typename F>
__device__ __forceinline__ void each(const T* data, bool wide, int from,
                                     int to, int t, int threads, F f) {
  constexpr int E = Vec<T>::E;
  int done = from;
  if (wide) {
    const int words = (to - from) / E;
    const uint4* p = reinterpret_cast<const uint4*>(data + from);
#pragma unroll 1
    for (int v = t; v < words; v += threads) {
      const Vec<T> x{p[v]};
#pragma unroll
      for (int k = 0; k < E; ++k) f(from + v * E + k, x.at(k));
    }
    done = from + words * E;
  }
  for (int i = done + t; i < to; i += threads) f(i, to_f32(data[i]));
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
// that is more than kCand, or more than kOwn of one.  `call`: a number not used before; a cluster
// barrier lies between the last use of all_cand and this.  What it wrote is
// there after it, and nothing of another CTA is read any more.
__device__ bool collect(Shared& S, cg::cluster_group& cl, int call, int* all) {
  __syncthreads();
  const int C = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x;
  const uint32_t mine = S.listed <= kOwn ? S.listed : kCand + 1;
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

__device__ __forceinline__ float x_of_word(u64 w, const Row& r) {
  return x_of(of_key((uint32_t)(w >> 32)), r);
}

// A range of words, in slots of equal width from the largest down.
struct Slots {
  u64 hi, lo;
  int shift;
  __device__ __forceinline__ Slots(u64 hi_, u64 lo_)
      : hi(hi_), lo(lo_) {
    // kSlots is 2^10; the float's exponent may be one more than the integer's
    const int e = (int)(__float_as_uint(__ull2float_rn(hi - lo)) >> 23) - 127;
    shift = max(0, e - 9);
  }
  __device__ __forceinline__ bool has(u64 w) const { return w >= lo && w <= hi; }
  __device__ __forceinline__ int of(u64 w) const {
    return (int)((hi - w) >> shift);
  }
  __device__ __forceinline__ Slots within(int slot) const {
    const u64 top = hi - ((u64)slot << shift);
    const u64 width = (1ull << shift) - 1;
    return Slots(top, top - lo > width ? top - width : lo);
  }
};
__device__ __forceinline__ void clear_slots(Shared& S) {
  for (int i = threadIdx.x; i < kSlots; i += kThreads)
    S.slots[i] = S.w_lo[i] = S.w_hi[i] = 0;
  if (threadIdx.x == 0) S.n_list = 0;
  __syncthreads();
}

// The cut among the n candidates (S.all_cand): of those with a key other than
// 0, in [lo, hi], by falling key the k-th, or the one whose weight makes the
// sum reach need_w(weight of all); S.cut is its key, S.kept_before the weight
// down to it.  Slots hold the candidates' numbers and weights; a scan finds
// the cut's slot, and comparing each with each finds it among the slot's few
// members (ties by the hundred make a range of their own, in finer slots).
// Returns 0 if the weight is not reached, 1 if the slots are those of [lo, hi]
// still (which `filled` tells the next call), else 2.  Whole CTA.
template <typename Key, typename Need>
__device__ int cut_in(Shared& S, const Row& r, int n, u64 hi, u64 lo,
                      bool filled, bool by_weight, uint32_t k, Key key,
                      Need need_w) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  Slots at(hi, lo);
  uint32_t n0 = 0;       // before the range
  u64 w0 = 0, need = 0;
  for (bool first = true;; first = false) {
    if (first && filled) {
      if (tid == 0) S.n_list = 0;
    } else {
      clear_slots(S);
      for (int i = tid; i < n; i += kThreads) {
        const u64 c = S.all_cand[i], w = key(c);
        if (w == 0 || !at.has(w)) continue;
        const int b = at.of(w);
        atomicAdd(&S.slots[b], 1u);
        add_weight(S, b, weight_of(x_of_word(c, r)));
      }
      __syncthreads();
    }
    find_bin<kSlots>(
        S, kSlots, [&](int i) { return S.slots[i]; },
        [&](int i) { return ((u64)S.w_hi[i] << 32) + S.w_lo[i]; }, by_weight,
        k - n0, [&](u64 all) { return first ? need_w(all) : need - w0; });
    const int slot = S.found_bin;
    if (first) need = S.target;
    if (slot < 0) {
      __syncthreads();
      return 0;
    }
    n0 += S.found_n;
    w0 += S.found_w;
    at = at.within(slot);
    u64 most = 0, least = ~0ull;
    for (int i = tid; i < n; i += kThreads) {
      const u64 c = S.all_cand[i], w = key(c);
      if (w == 0 || !at.has(w)) continue;
      const uint32_t to = atomicAdd(&S.n_list, 1u);
      if (to < kList) {
        S.list[to] = w;
        S.list_w[to] = weight_of(x_of_word(c, r));
      }
      most = max(most, w);
      least = min(least, w);
    }
    __syncthreads();
    const int m = (int)S.n_list;
    if (m <= kList) {
      if (tid < m) {
        const u64 mine = S.list[tid], w = S.list_w[tid];
        uint32_t rank = n0;
        u64 before = w0;
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
      return first ? 1 : 2;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    }
    if (lane == 0) {
      S.list[wid] = most;
      S.list[kWarps + wid] = least;
    }
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
      most = max(most, S.list[i]);
      least = min(least, S.list[kWarps + i]);
    }
    if (most == least) {  // no finer slots part them (no two tokens' keys are
      __syncthreads();    // equal: this bounds the loop whatever is there)
      if (tid == 0) {
        S.cut = most;
        S.kept_before = w0;
      }
      __syncthreads();
      return 2;
    }
    at = Slots(most, least);
  }
}

// The row's n candidates (its largest tokens, none below `low`, at least k of
// them) to the kept set's cut and size, and the token.  The first k are kept,
// of those the ones whose predecessors weigh less than `bound` (0: p of the k
// tokens' weight).  Whole CTA.  A lone row of 151936 logits: k = 1000, p = 0.9
// (1053 candidates) 19 us, k = 50 13 us; with two sorts of the candidates (by
// rank, then by id) 41 us and 21 us.
__device__ void pick(Shared& S, const Row& r, float low, int V, int n, int k,
                     u64 bound, float p, float mp, float u, int* token) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    S.kept = 0;
    S.least_key = ~0u;
  }
  const u64 hi = (u64)key_of(r.top) << 32 | 0xffffffffu;
  const u64 lo = (u64)key_of(low) << 32;
  auto whole = [](u64 c) { return c; };
  const bool found =
      bound && cut_in(S, r, n, hi, lo, false, true, 0, whole,
                      [&](u64) { return bound; });
  if (!found) {  // all are lighter, if there is a bound
    const int filled = cut_in(S, r, n, hi, lo, bound != 0, false, (uint32_t)k,
                              whole, [](u64) { return 0ull; });
    if (bound == 0 && p < 1.f) {
      const u64 need = top_p_bound(p, S.kept_before);
      cut_in(S, r, n, hi, lo, filled == 1, true, 0, whole,
             [&](u64) { return need; });
    }
  }
  const u64 cut = S.cut;
  auto keeps = [&](u64 c) {
    return c >= cut && (mp == 0.f || x_of_word(c, r) >= mp);
  };
  for (int i = tid; i < n; i += kThreads) {
    const u64 c = S.all_cand[i];
    if (!keeps(c)) continue;
    atomicAdd(&S.kept, 1);
    if (mp > 0.f) atomicMin(&S.least_key, (uint32_t)(c >> 32));
  }
  // the kept tokens by id: the word's lower half is the id's complement
  cut_in(S, r, n, 0xffffffffu, (uint32_t)~(uint32_t)(V - 1), false, true, 0,
         [&](u64 c) { return keeps(c) ? (u64)(uint32_t)c : 0ull; },
         [&](u64 all) { return draw_target(u, all) + 1; });
  if (tid == 0) {
    *token = (int)~(uint32_t)S.cut;
    // what is kept, as one cut: all of the smallest logit if min-p decided
    S.cut = mp > 0.f ? max(cut, (u64)S.least_key << 32 | 0x80000000u) : cut;
  }
}

// The row's cut where nothing narrows it: slots over the words of all tokens,
// then over the cut's slot, until its members fit a list.
template <typename T>
__device__ void refine_cut(Shared& S, cg::cluster_group& cl, const T* data,
                           bool wide, int n, int id0, const Row& r, int call,
                           bool by_weight, uint32_t need_n, u64 need_w) {
  const int tid = threadIdx.x;
  Slots at(~0ull, 0);
  uint32_t n0 = 0;  // before the range
  u64 w0 = 0;
  for (;;) {
    clear_slots(S);
    each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
      const u64 w = word_of(l, id0 + i);
      if (!(l > -INFINITY) || !at.has(w)) return;
      const int b = at.of(w);
      atomicAdd(&S.slots[b], 1u);
      add_weight(S, b, weight_of(x_of(l, r)));
    });
    cl.sync();
    for (int i = tid; i < kSlots; i += kThreads) {
      uint32_t c = 0;
      u64 w = 0;
      for (int q = 0; q < cl.num_blocks(); ++q) {
        const Shared* o = cl.map_shared_rank(&S, q);
        c += o->slots[i];
        w += ((u64)o->w_hi[i] << 32) + o->w_lo[i];
      }
      S.all_n[i] = c;
      S.all_w[i] = w;
    }
    cl.sync();
    find_bin<kSlots>(S, kSlots, [&](int i) { return S.all_n[i]; },
                     [&](int i) { return S.all_w[i]; }, by_weight,
                     need_n - n0, [&](u64) { return need_w - w0; });
    const int slot = S.found_bin;
    if (slot < 0) {  // no cut (the caller has counted: this does not happen)
      __syncthreads();
      if (tid == 0) {
        S.cut = 0;
        S.kept_before = w0;
      }
      __syncthreads();
      return;
    }
    n0 += S.found_n;
    w0 += S.found_w;
    at = at.within(slot);
    if (S.all_n[slot] <= kOwn) break;
    __syncthreads();
  }
  if (tid == 0) S.listed = 0;
  cl.sync();  // the first CTA's sums are where the list will be
  each(data, wide, 0, n, tid, kThreads, [&](int i, float l) {
    const u64 w = word_of(l, id0 + i);
    if (!(l > -INFINITY) || !at.has(w)) return;
    const uint32_t to = atomicAdd(&S.listed, 1u);
    if (to < kOwn) S.cand[to] = w;
  });
  int all;
  collect(S, cl, call, &all);
  if (cl.block_rank() == 0) {
    cut_in(S, r, min(all, kCand), at.hi, at.lo, false, by_weight, need_n - n0,
           [](u64 c) { return c; }, [&](u64) { return need_w - w0; });
    const u64 cut = S.cut, before = w0 + S.kept_before;
    __syncthreads();
    if (tid < cl.num_blocks()) {
      Shared* o = cl.map_shared_rank(&S, tid);
      o->cut = cut;
      o->kept_before = before;
    }
  }
  cl.sync();
}

// Three CTAs to an SM (40 registers each thread) hide each other's barriers:
// 288 rows with mixed filters and filtered logits 160 us, 169 us with two (64
// registers).  Where there are no more than two to an SM, 64 registers spare the
// spills: 64 rows with top-p 0.9 54 us, 71 us with 40 registers.
template <typename T, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm)
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
  // A thread's tokens are four quarters: of a slice that is copied, a quarter
  // of each copy's words, else every fourth of its words (or tokens).
  constexpr int E = Vec<T>::E;
  const int words = n / E, per = (words + kChunks - 1) / kChunks;

  // ---- the slice and the row's maximum -------------------------------------
  if (tid == 0) {
    S.odd = S.fine = S.late = 0;
    S.kept_n = 0;
    S.cut = 0;
    S.listed = S.n_quarters = 0;
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
  uint32_t bits = 0;
  auto take = [&](int c, float l) {
    odd |= !(fabsf(l) < INFINITY);
    bits |= __float_as_uint(l);
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
      tc::mbar_wait_bounded(&S.landed[c], 0, &give_up, a.wait_ns);
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
    if (give_up) {  // the row is, but not while a copy is in flight
      S.late = 1;
      int never = 0;
#pragma unroll 1
      for (int c = 0; c < kChunks; ++c)
        tc::mbar_wait_bounded(&S.landed[c], 0, &never, kWaitLimitNs);
    }
  } else if (src_wide) {
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
  if (bits & 0xffffu) S.fine = 1;
  if (tid == 0) {
    for (int i = 1; i < kWarps; ++i)
      top = fmaxf(top, __uint_as_float((uint32_t)S.warp_w[i]));
    if (S.late) {
      raise_error(a.err, kErrTimeout);
      top = NAN;
    }
    S.top = top;
  }
  cl.sync();
  top = lane < C ? cl.map_shared_rank(&S, lane)->top : -INFINITY;
  if (__any_sync(0xffffffffu, top != top)) {  // uniform over the cluster
    if (rank == 0 && tid == 0) {
      a.token[row] = -1;
      if (a.n_kept) a.n_kept[row] = 0;
    }
    cl.sync();  // no CTA leaves while another reads its maximum
    return;
  }
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
  const float p = S.top_p < 0.f ? 0.f : S.top_p;
  // at most 1 (which keeps the maximum), 0 for what is no number
  const float mp = S.min_p > 0.f ? fminf(S.min_p, 1.f) : 0.f;
  const float u = S.u;
  const bool by_k = !r.greedy && !empty && k > 0 && k < a.V;
  const bool by_p = !r.greedy && !empty && p < 1.f;
  // f(i, logit) over the slice's tokens from `low` up: those of the threads'
  // quarters whose maximum is not below it, a word to a thread.  Once a row.
  auto from = [&](float low, auto f) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (tops[c] >= low && tops[c] > -INFINITY)
        S.quarters[atomicAdd(&S.n_quarters, 1u)] = c * kThreads + tid;
    __syncthreads();
    const bool copied = a.resident && src_wide;
    const int step = copied ? kThreads : kChunks * kThreads;
    const int units = src_wide ? words : n;  // words, or tokens
    const uint32_t q = (copied ? per + step - 1 : units + step - 1) / step;
    const uint32_t items = S.n_quarters * q;
    auto test = [&](int i, float l) {
      if (l >= low && l > -INFINITY) f(i, l);
    };
#pragma unroll 2
    for (uint32_t it = tid; it < items; it += kThreads) {
      const uint32_t at = it / q;
      const int of = S.quarters[at], c = of / kThreads;
      int v = of + (int)(it - at * q) * step, to = units;
      if (copied) {
        v += c * (per - kThreads);
        to = min(words, (c + 1) * per);
      }
      if (v >= to) continue;
      if (src_wide) {
        const Vec<T> x{reinterpret_cast<const uint4*>(data)[v]};
#pragma unroll
        for (int k = 0; k < E; ++k) test(v * E + k, x.at(k));
      } else {
        test(v, to_f32(data[v]));
      }
    }
    if (src_wide)
      for (int i = words * E + tid; i < n; i += kThreads)
        test(i, to_f32(data[i]));
  };
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
        __stcs(reinterpret_cast<float4*>(dst) + v,
               make_float4(f[0], f[1], f[2], f[3]));
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
      from(top, [&](int i, float) { first = min(first, id0 + i); });
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
  // CTA; false if they are too many.  At most once a row: neither the places
  // that collect() gave out nor the quarters of from() are taken back.
  auto finish = [&](float low, int most, u64 bound) {
    from(low, [&](int i, float l) {
      const uint32_t at = atomicAdd(&S.listed, 1u);
      if (at < kOwn) S.cand[at] = word_of(l, id0 + i);
    });
    int all;
    if (!collect(S, cl, 0, &all)) return false;
    if (rank == 0) {
      pick(S, r, low, a.V, all, min(most, all), bound, p, mp, u,
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
    find_bin<kCandBins>(S, kCandBins, [&](int i) { return of[i]; },
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
    if (finish(low, k, 0)) return;
  }

  // ---- the cut by counts in bins ----------------------------------------------
  const bool by_m = mp > 0.f;
  const float low_m =  // no token kept by min-p is below
      by_m ? weight_floor(mp, r, t) : -INFINITY;
  // min-p alone: its tokens, if they are few, are candidates of no other bound
  if (by_m && !by_k && !by_p && finish(low_m, kCand, ~0ull)) return;
  u64 cut = 0;
  bool done = false;  // kept_w and kept_n are those of the cut

  // The tokens of bins [0, bins) from `low` up into the bins, over the
  // cluster; the weight of all tokens, and of those in the first kTopBins.
  auto fill = [&](float low, int bins, u64* top_w) {
    for (int i = tid; i < bins; i += kThreads) S.count[i] = 0;
    if (tid < 32) S.w_lo[tid] = S.w_hi[tid] = 0;
    __syncthreads();
    u64 sum = 0;
    if (!S.odd && r.inv_t < INFINITY) {  // as in the sum of all weights below
      for (int b = 0; b < n; b += kThreads * kBlock) {
        uint32_t hi = 0, lo = 0, m = 0;
        each(data, wide, b, min(n, b + kThreads * kBlock), tid, kThreads,
             [&](int, float l) {
               const float z = __fmul_rn(__fsub_rn(l, r.top), r.inv_t);
               const WeightBits w = weight_bits(expf(z));
               hi += w.hi;
               lo += w.lo;
               ++m;
               // (the integer part by an addition to 2^23, as in weight_bits)
               const float b = __fmaf_rz(z, -kBinsPerUnit, 0x1p23f);
               const uint32_t bin = __float_as_uint(b) - 0x4b000000u;
               if (l >= low) atomicAdd(&S.count[min(bin, bins - 1u)], 1u);
               if (bin < kTopBins)
                 add_weight(S, lane,
                            (u64)(w.hi - 0x4b000000u) * (1u << 23) +
                                (w.lo - 0x4b000000u));
             });
        sum += (u64)(hi - m * 0x4b000000u) * (1u << 23) +
               (lo - m * 0x4b000000u);
      }
    } else {
      each(data, wide, 0, n, tid, kThreads, [&](int, float l) {
        if (!(l > -INFINITY)) return;
        const u64 w = weight_of(x_of(l, r));
        const int bin = bin_of(l, r);
        sum += w;
        if (l >= low) atomicAdd(&S.count[min(bin, bins - 1)], 1u);
        if (bin < kTopBins) add_weight(S, lane, w);
      });
    }
    sum = warp_total(sum);
    if (lane == 0) S.warp_w[wid] = sum;
    __syncthreads();
    if (wid == 0) {
      sum = warp_total(lane < kWarps ? S.warp_w[lane] : 0ull);
      const u64 tw = warp_total(((u64)S.w_hi[lane] << 32) + S.w_lo[lane]);
      if (lane == 0) {
        S.total = sum;
        S.top_w = tw;
      }
    }
    reduce_counts(S, cl, bins);
    u64 total = 0;
    *top_w = 0;
    for (int c = 0; c < C; ++c) {
      total += cl.map_shared_rank(&S, c)->total;
      *top_w += cl.map_shared_rank(&S, c)->top_w;
    }
    return total;
  };

  // The cut if it lies in [lo, hi]: kept_w and kept_n of the tokens above, the
  // others listed, cut, and counted if kept.  False if it does not, or if
  // there are too many of them.
  auto narrow = [&](int call, float lo, float hi, bool by_weight,
                    uint32_t need_n, u64 need_w) {
    if (tid == 0) {
      S.listed = 0;
      S.kept_n = 0;
      S.cut = 0;
    }
    __syncthreads();
    int c0, c1;
    warp_chunk(n, wid, &c0, &c1);
    u64 sum = 0;
    uint32_t cnt = 0;
    for (int b = c0; b < c1; b += 32 * kBlock) {  // as in all weights' sum
      uint32_t w_hi = 0, w_lo = 0, m = 0;
      each(data, wide, b, min(c1, b + 32 * kBlock), lane, 32,
           [&](int i, float l) {
             const bool on = l > hi;
             const WeightBits w = weight_bits(on ? x_of(l, r) : 0.f);
             w_hi += w.hi;
             w_lo += w.lo;
             ++m;
             cnt += on;
             if (l >= lo && !on && l > -INFINITY) {
               const uint32_t at = atomicAdd(&S.listed, 1u);
               if (at < kOwn) S.cand[at] = word_of(l, id0 + i);
             }
           });
      sum += (u64)(w_hi - m * 0x4b000000u) * (1u << 23) +
             (w_lo - m * 0x4b000000u);
    }
    sum = warp_total(sum);
    cnt = warp_total(cnt);
    if (lane == 0) {
      S.kept_w[wid] = sum;
      if (cnt) atomicAdd(&S.kept_n, cnt);
    }
    int all;
    if (!collect(S, cl, call, &all)) return false;
    if (rank == 0) {
      sum = 0;
      for (int i = lane; i < C * kWarps; i += 32)
        sum += cl.map_shared_rank(&S, i / kWarps)->kept_w[i % kWarps];
      sum = warp_total(sum);
      cnt = warp_total(lane < C ? cl.map_shared_rank(&S, lane)->kept_n : 0u);
      if (by_weight ? sum < need_w : cnt < need_n) {  // uniform
        cut_in(S, r, all, (u64)key_of(hi) << 32 | 0xffffffffu,
               (u64)key_of(lo) << 32, false, by_weight, need_n - cnt,
               [](u64 c) { return c; }, [&](u64) { return need_w - sum; });
        const u64 at_cut = S.cut, before = sum + S.kept_before;
        __syncthreads();
        if (tid < C) {
          Shared* o = cl.map_shared_rank(&S, tid);
          o->cut = at_cut;
          o->kept_before = before;
        }
      }
    }
    cl.sync();
    const u64 at_cut = S.cut;
    if (at_cut == 0) return false;
    // (the first CTA's slots have overwritten its list)
    const u64* mine = rank == 0 ? S.all_cand + S.list_at : S.cand;
    const int per = ((n + kWarps - 1) / kWarps + 127) & ~127;
    for (uint32_t i = tid; i < S.listed; i += kThreads) {
      const u64 c = mine[i];
      if (c < at_cut) continue;
      atomicAdd(&S.kept_w[((int)~(uint32_t)c - id0) / per],
                weight_of(x_of_word(c, r)));
      atomicAdd(&S.kept_n, 1u);
    }
    __syncthreads();
    return true;
  };

  u64 total = 0, top_w;
  bool have_total = false;
  if (by_k) {
    fill(-INFINITY, kBins, &top_w);
    find_bin<kBins>(S, kBins, [&](int i) { return S.all_count[i]; },
             [](int) { return 0ull; }, false, (uint32_t)k,
             [](u64) { return 0ull; });
    const int bin = S.found_bin;
    __syncthreads();
    if (bin >= 0) {  // fewer than k tokens above -inf: no cut
      done = narrow(1, bin_floor(bin, r, t), bin_ceil(bin, r, t), false,
                    (uint32_t)k, 0);
      if (!done)
        refine_cut(S, cl, data, wide, n, id0, r, 3, false, (uint32_t)k, 0);
      cut = S.cut;
      total = S.kept_before;
      have_total = true;
      __syncthreads();
    }
  }
  if (by_p) {
    // Tokens of less than (1 - p) W / V weigh less than (1 - p) W together, so
    // they are past the cut and need no bin.  The weight of this CTA's
    // threads' maxima, times 0.9 for roundings, stands for W from below where
    // no top-k has a say; 1 does for all CTAs, and for how many bins they use.
    float sum = 0.f;
    if (!by_k) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
        if (tops[c] > -INFINITY) sum += x_of(tops[c], r);
      sum = warp_sum(sum);
      if (lane == 0) S.warp_n[wid] = __float_as_uint(sum);
      __syncthreads();
      sum = 0.f;
      for (int i = 0; i < kWarps; ++i) sum += __uint_as_float(S.warp_n[i]);
      __syncthreads();
    }
    const float share = 0.9f * (1.f - p) / (float)a.V;
    const float least_x = share * fmaxf(sum, 1.f);
    const float low =
        fmaxf(least_x > 0.f && least_x < 1.f ? weight_floor(least_x, r, t)
                                             : -INFINITY, low_m);
    const int bins =
        share > 0.f
            ? min(kBins, (int)(-logf(share) * kBinsPerUnit * 1.001f) + 3)
            : kBins;
    const u64 weight = fill(low, bins, &top_w);
    const u64 bound = top_p_bound(p, have_total ? total : weight);
    auto count = [&](int i) { return S.all_count[i]; };
    // The bin of the cut.  A bin's tokens all weigh that of its place `at`;
    // the first bins, whose tokens are few and heavy, weigh what they do if
    // the cut is past them: a token of weight w puts the sum off by w / 128 at
    // most, of which the cut's own bin may hold less.  (The last may hold
    // tokens of beyond it: nothing, from below.)
    // Logits that are bf16 numbers do not fill a bin evenly: they all stand at
    // the one that is next to its middle.
    const u64 off = bound > top_w ? top_w : 0;
    bool coarse = true;
    for (int c = 0; c < C; ++c) coarse &= !cl.map_shared_rank(&S, c)->fine;
    auto find = [&](float at, float slack) {
      find_bin<kBins>(S, bins, count,
               [&](int i) {
                 float x = expf(((float)i + at) * (-1.f / kBinsPerUnit));
                 if (coarse && slack == 0.f) {
                   const float l = __bfloat162float(__float2bfloat16_rn(
                       r.top - ((float)i + at) * t * (1.f / kBinsPerUnit)));
                   if (l <= r.top && bin_of(l, r) == i) x = x_of(l, r);
                 }
                 const float w = floorf(x * 0x1p44f * (1.f + slack)) +
                                 (slack < 0.f ? -1.f : 1.f);
                 return (slack < 0.f && i == bins - 1) || (off && i < kTopBins)
                            ? 0ull
                            : S.all_count[i] * (u64)fmaxf(w, 0.f);
               },
               true, 0, [&](u64) { return bound - off; });
      return S.found_bin;
    };
    int bin = find(0.5f, 0.f);
    // (with a top-k, whose tokens finish() may have listed already: no second
    // time)
    if (!by_k && bin >= 0 && S.found_n + S.all_count[bin] <= kOwn * 3 / 4) {
      __syncthreads();
      const int last = find(1.f, -1e-4f);  // from below: the cut is not past it
      if (last >= 0 && S.found_n + S.all_count[last] <= kOwn * 7 / 8) {
        if (tid == 0) S.listed = 0;
        __syncthreads();
        if (finish(bin_floor(last, r, t), kCand, bound)) return;
        fill(low, bins, &top_w);  // the list has overwritten the bins
      }
    }
    __syncthreads();
    bool past = false;  // the cut is past all tokens that min-p keeps
    if (by_m && bin < 0) {
      past = find(0.f, 1e-4f) < 0;
      __syncthreads();
    }
    if (!past) {
      if (bin < 0) bin = bins - 1;
      // one bin on each side of it, more while they hold few tokens
      int b0 = bin, b1 = bin;
      uint32_t c = S.all_count[bin];
      for (int i = 0; i < 16 && (i < 2 || c < 512); ++i) {
        const int b = i & 1 ? b0 - 1 : b1 + 1;
        if (b < 0 || b >= bins || c + S.all_count[b] > kOwn - 128) continue;
        c += S.all_count[b];
        b0 = min(b0, b);
        b1 = max(b1, b);
      }
      __syncthreads();
      done = narrow(2, bin_floor(b1, r, t), bin_ceil(b0, r, t), true, 0, bound);
      if (!done)
        refine_cut(S, cl, data, wide, n, id0, r, 4, true, 0, bound);
      cut = max(cut, S.cut);
      __syncthreads();
    }
  }
  done = done && !by_m;
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
  if (done) {
    // (there already)
  } else if (cut == 0 && !by_m) {
    if (S.odd || !(r.inv_t < INFINITY)) {  // uniform in the CTA
      each(data, wide, c0, c1, lane, 32, [&](int, float l) {
        const bool on = l > -INFINITY;  // not a NaN, either
        sum += weight_of(on ? x_of(l, r) : 0.f);
        cnt += on;
      });
    } else {
      // All weights are wanted and all logits finite.  The 0x4b000000 of
      // every float comes off at the end.
      for (int b = c0; b < c1; b += 32 * kBlock) {
        const int e = min(c1, b + 32 * kBlock);
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
        fmaxf(cut ? of_key((uint32_t)(cut >> 32)) : -INFINITY, low_m);
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
  if (!done) {
    if (tid == 0) S.kept_n = 0;
    __syncthreads();
    if (lane == 0) {
      S.kept_w[wid] = sum;
      S.kept_least[wid] = least;
      if (cnt) atomicAdd(&S.kept_n, cnt);
    }
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
    const u64 all = __shfl_sync(0xffffffffu, run, 31);
    if (rank == 0) {
      uint32_t nk = lane < C ? cl.map_shared_rank(&S, lane)->kept_n : 0;
      nk = warp_total(nk);
      if (lane == 0 && a.n_kept) a.n_kept[row] = (int)nk;
    }
    const u64 target = draw_target(u, all);
    u64 before = run - mine;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (target >= before && target < before + w[j]) {
        S.found_bin = lane * kPer + j;
        S.target = target - before;  // within the chunk
      }
      before += w[j];
    }
  }
  __syncthreads();
  const int chunk = S.found_bin;
  if (chunk / kWarps == rank) {  // it is in this CTA's slice
    u64 target = S.target;
    warp_chunk(n, chunk % kWarps, &c0, &c1);
    auto weight_at = [&](int i) {
      const float l = to_f32(data[i]);
      const float x = x_of(l, r);
      return keeps(l, i, x) ? weight_of(x) : 0;
    };
    const int each_n = (c1 - c0 + kThreads - 1) / kThreads;
    const int i0 = c0 + tid * each_n, i1 = min(c1, i0 + each_n);
    u64 mine = 0, all;
    for (int i = i0; i < i1; ++i) mine += weight_at(i);
    u64 at = cta_scan(S, mine, &all);
    if (target >= at && target < at + mine)
      for (int i = i0; i < i1; ++i) {
        const u64 w = weight_at(i);
        if (target >= at && target < at + w) a.token[row] = id0 + i;
        at += w;
      }
  }
  cl.sync();  // no CTA leaves while another reads its sums
}

template <typename T>
cudaError_t launch(SampleArgs a, int sms, cudaStream_t s) {
  // One wave of CTAs, three to an SM: fewer to a row cost less in barriers
  // between them (64 rows of 262144 bf16 logits in L2, top-k 50: 17 us with
  // four, 27 us with eight; a lone row without filters 10 us with eight, 24 us
  // with two).  But no slices of more than 65536 tokens, up to eight CTAs for
  // each SM: rows differ in how long they take, and in several waves the short
  // ones fill what the long ones leave (288 rows of 151936 with mixed filters:
  // 160 us with four, 261 us with one; with top-k 50 in all of them 60 us and 43
  // us).  Never more than slices of 4096 tokens need.
  int C = kMaxCluster;
  while (C > 1 && ((long long)a.R * C > 3 * sms ||
                   (long long)(C / 2) * 4096 >= a.V))
    C /= 2;
  while (C < kMaxCluster && (long long)C * 65536 < a.V &&
         (long long)a.R * C * 2 <= 8 * sms)
    C *= 2;
  // A slice stays in shared memory where that takes no CTA's place on an SM
  // (100 rows of 151936 logits in L2, top-k 50: 23 us, with slices of 148 KB
  // held, one CTA to an SM, 35 us); the rest is read again, from L2 for the most
  // part.
  const bool two = (long long)a.R * C <= 2 * sms;
  a.slice = (int)((((long long)a.V + C - 1) / C + 7) & ~7ll);
  a.resident =
      (long long)a.slice * (long long)sizeof(T) <= (two ? 76 : 36) * 1024;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 +
                      (a.resident ? (size_t)a.slice * sizeof(T) : 16);
  auto* f = two ? sample_kernel<T, 2> : sample_kernel<T, 3>;
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
  if (R < 1 || R > (1 << 24) || V < 1 || V >= (1 << 20)) return 0;
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
  a.wait_ns = wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == DFLASH_FP32
                            ? launch<float>(a, sms, s)
                            : launch<__nv_bfloat16>(a, sms, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
