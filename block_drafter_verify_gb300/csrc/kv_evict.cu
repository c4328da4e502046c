// Eviction from the paged 8-bit cache by the attention weight that tokens have
// gathered.
//
// Mathematics.  Of a key head's n > budget slots the first `sink` and the last
// `recent` stay, and of the others the budget - sink - recent of largest weight
// (ties: the lower slot).  That is a cut in the order of 32-bit keys, found by
// three histograms (11, 11 and 10 bits), and the first few of the slots that
// lie on it.  The kept slots move to slots 0 .. budget - 1 in their order.  A
// page that gets other tokens gets a scale of its own, the least power of two
// with max |x| <= 448 s, as an append would give it: codes move exactly but for
// those that become subnormal.
//
// One launch: a CTA for every sequence and key head, or a cluster of up to
// eight where there are few.  It finds the cut (a thread holds the weights of
// 16 slots in registers over the histograms), writes the list of kept slots,
// and moves their codes, in place: slots only move down, so pages are taken in
// rounds, lower ones first, of as many as the cluster's warps hold in
// registers.  A round's pages are all read, the cluster meets, and they are
// written: what a later round reads lies above.
//
// What bounds it: with few heads the chain of steps (three histograms, then the
// loads of a round; kept slots and page ids are asked for a round ahead), with
// many bytes.  Eight heads of 128: 2100 to 2048 tokens 20 us, 131072 to 100000
// tokens 255 us; 32 such sequences of up to 8000 tokens to 6000 at most 123 us
// (59 us of bytes at the copy's rate; half of the issue slots: some 170
// instructions for 16 codes, most of them maxima and conversions), where a
// launch for the lists, one for the codes and whole histograms took 193 us, and
// pages in any order, each waiting for flags of those that read it, 170 us.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "kernels.h"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

namespace cg = cooperative_groups;

constexpr int kMinExp = -64;      // smallest exponent of a block scale
constexpr int kBins = 2048;
constexpr int kGroups = 64;       // of 32 bins
constexpr int kEach = 4;          // consecutive slots of a thread
constexpr int kTimes = 4;         // and how often, in registers
constexpr int kMaxCluster = 8;

struct EvictArgs {
  const float* mass;
  long long ld_mass, ld_out;      // slots of a head in mass and mass_out
  uint8_t* codes[2];
  float* scale[2];
  const int *table, *kv_len;
  int B, Hkv, D, page, num_pages, max_pages, budget, sink, recent;
  float* mass_out;                // may be NULL
  int *new_len, *kept;
  int* err;
};

// Order-preserving key (equal for -0 and 0); a NaN is below all numbers.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0;
  const uint32_t w = __float_as_uint(x + 0.f);
  return w & 0x80000000u ? ~w : w | 0x80000000u;
}

__device__ __forceinline__ int length_of(const EvictArgs& a, int b,
                                         bool* bad) {
  return attn_clamp(a.kv_len[b],
                    min((long long)a.max_pages * a.page, a.ld_mass), bad);
}

// Exponent of the least power of two s with x <= 448 s, x the value of an E4M3
// code without its sign: 448 is 1.75 2^8, and a code's largest fraction is
// 1.875.
__device__ __forceinline__ int scale_exponent(uint32_t code) {
  if (code < 8)                              // 0, or 1 to 7 times 2^-9
    return code == 0 ? -1000 : 31 - __clz((int)code) - 17;
  return (int)(code >> 3) - 15 + ((code & 7) == 7);
}
// The largest of a unit's 16 codes without their signs.
__device__ __forceinline__ uint32_t largest(const uint4& w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;                            // of even and of odd bytes
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __vmaxu2(m, __vmaxu2(x[i] & 0x007f007fu, x[i] >> 8 & 0x007f007fu));
  return max(m & 0xffffu, m >> 16);
}
// Four codes times 2^off, rounded to codes again.  In fp16, which has room for
// what a code times 2^-11 to 2^7 needs; else in fp32.  (Below 2^-40 a code is
// 0, above 2^17 all of them are: the scale is made for the largest.)
__device__ __forceinline__ uint32_t requant4(uint32_t w, int off) {
  uint32_t out = 0;
  if (off >= -11 && off <= 7) {
    const __half2 up = __half2half2(
        __ushort_as_half((unsigned short)((off + 15) << 10)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 h = __hmul2(
          __half2(__nv_cvt_fp8x2_to_halfraw2(
              (__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3)), up);
      out |= (uint32_t)__nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3)
             << (16 * i);
    }
  } else {
    const float ratio =
        __uint_as_float((uint32_t)(min(max(off, -40), 40) + 127) << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
          (__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3)));
      out |= (uint32_t)__nv_cvt_float2_to_fp8x2(
                 make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE,
                 __NV_E4M3)
             << (16 * i);
    }
  }
  return out;
}

template <int kWarps>
struct alignas(16) Shared {
  int hist[kBins];
  int group[kGroups];                        // its sums
  int sum[kMaxCluster][kGroups];             // of every CTA of the cluster
  int warp_n[2][kWarps];
  int n_gt[kMaxCluster], n_eq[kMaxCluster];  // of every CTA of the cluster
  int stay;                                  // pages that stay as they are
  int exp[2][kWarps];
};

// kOf warps have a page, kUnits 16-byte units of its keys and of its values a
// lane.
template <int kThreads, int kOf, int kUnits>
__global__ void __launch_bounds__(
    kThreads, kThreads == 512 ? 1 : kUnits == 4 ? 4 : 2)
    kv_evict_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kHeld = kThreads * kEach * kTimes;
  constexpr int kOwn = kBins / kThreads;     // bins of a thread
  __shared__ Shared<kWarps> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  pdl_trigger();
  pdl_wait();
  const int item = blockIdx.x / C;
  const int h = item % a.Hkv, b = item / a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * a.Hkv + h;
  bool bad = false;
  const int n = length_of(a, b, &bad);
  const float* mass = a.mass + bh * a.ld_mass;
  float* mass_out = a.mass_out ? a.mass_out + bh * a.ld_out : nullptr;
  int* kept = a.kept + bh * a.budget;
  if (h == 0 && me == 0 && tid == 0) {
    a.new_len[b] = min(n, a.budget);
    if (bad) raise_error(a.err, kErrBadIndex);
  }
  if (n <= a.budget) {             // (the same in the whole cluster)
    for (int i = me * kThreads + tid; i < a.budget; i += C * kThreads)
      kept[i] = i < n ? i : -1;
    if (mass_out)
      for (int i = me * kThreads + tid; i < n; i += C * kThreads)
        mass_out[i] = mass[i];
    return;
  }
  // (n > budget >= sink + recent: the two ends do not meet)
  const int lo = a.sink, hi = n - a.recent;
  const int want = a.budget - a.sink - a.recent;
  // this CTA's slots, in multiples of a thread's
  const int per = (n + C * kEach - 1) / (C * kEach) * kEach;
  const int s0 = min(n, me * per), s1 = min(n, s0 + per);
  const bool wide = a.ld_mass % 4 == 0 &&
                    (reinterpret_cast<uintptr_t>(a.mass) & 15) == 0;
  // kTimes * kEach slots of this thread from slot `from` on: slot (k, j) is
  // from + (k kThreads + tid) kEach + j
  float x[kTimes][kEach];
  auto load = [&](int from) {
#pragma unroll
    for (int k = 0; k < kTimes; ++k) {
      const int i = from + (k * kThreads + tid) * kEach;
      if (wide && i + kEach <= s1) {
        const float4 v = *reinterpret_cast<const float4*>(mass + i);
        x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          x[k][j] = i + j < s1 ? mass[i + j] : 0.f;
      }
    }
  };
  const bool held = s1 - s0 <= kHeld;
  if (held) load(s0);
  // ---- the cut: of the slots [lo, hi) those above `key`, and `left` on it
  uint32_t key = 0xffffffffu;
  int left = 0;
  if (want > 0) {
    uint32_t prefix = 0;
    left = want;
    bool nan = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int from = s0; from < s1; from += kHeld) {
        if (!held) load(from);
#pragma unroll
        for (int k = 0; k < kTimes; ++k)
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = from + (k * kThreads + tid) * kEach + j;
            if (i < lo || i >= min(hi, s1)) continue;
            const uint32_t w = key_of(x[k][j]);
            nan |= w == 0;
            if (pass == 0 || (w >> (shift + bits)) == prefix)
              atomicAdd(&sh.hist[(w >> shift) & ((1 << bits) - 1)], 1);
          }
      }
      // The bin, counted from the largest, in which the left-th slot lies:
      // first its group of 32, from the CTAs' sums of groups, then the bin.
      // (Whole histograms read from eight CTAs: 9000 cycles.)
      __syncthreads();
      {
        int n_own = 0;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) n_own += sh.hist[tid * kOwn + k];
        constexpr int kLanes = 32 / kOwn;    // of a group
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1)
          n_own += __shfl_xor_sync(0xffffffffu, n_own, o);
        if (tid % kLanes == 0) sh.group[tid / kLanes] = n_own;
      }
      if (C > 1) cluster.sync(); else __syncthreads();
      for (int i = tid; i < C * kGroups; i += kThreads)
        sh.sum[i / kGroups][i % kGroups] =
            (C > 1 ? cluster.map_shared_rank(sh.group, i / kGroups)
                   : sh.group)[i % kGroups];
      __syncthreads();
      // (largest first; every warp for itself)
      const int groups = (1 << bits) / 32;
      int group = 0, before = 0;             // slots in larger groups
      {
        int c[2] = {0, 0};
        const int g0 = groups - 1 - 2 * lane;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (g0 - k >= 0)
            for (int r = 0; r < C; ++r) c[k] += sh.sum[r][g0 - k];
        int run = c[0] + c[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += v;
        }
        const int above = run - c[0] - c[1];
        const bool in = above < left && left <= run;
        const bool second = left > above + c[0];
        const int from = __ffs(__ballot_sync(0xffffffffu, in)) - 1;
        group = __shfl_sync(0xffffffffu, g0 - (second ? 1 : 0), from);
        before = __shfl_sync(0xffffffffu, above + (second ? c[0] : 0), from);
      }
      __syncthreads();                       // (the sums have been read)
      if (warp < C)
        sh.sum[warp][lane] =
            (C > 1 ? cluster.map_shared_rank(sh.hist, warp)
                   : sh.hist)[group * 32 + lane];
      __syncthreads();
      {
        const int bin = group * 32 + 31 - lane;
        int c = 0;
        for (int r = 0; r < C; ++r) c += sh.sum[r][31 - lane];
        int run = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, run, o);
          if (lane >= o) run += v;
        }
        const int above = before + run - c;
        const int from = __ffs(__ballot_sync(
            0xffffffffu, above < left && left <= above + c)) - 1;
        prefix = prefix << bits |
                 (uint32_t)__shfl_sync(0xffffffffu, bin, from);
        left -= __shfl_sync(0xffffffffu, above, from);
      }
      // (the others have read this histogram before it is cleared)
      if (C > 1) cluster.sync(); else __syncthreads();
    }
    key = prefix;
    if (nan) raise_error(a.err, kErrNonfinite);
  } else if (C > 1) {
    cluster.sync();                          // (all CTAs have started)
  }
  // ---- the kept slots in their order ---------------------------------------
  // bit (k, j) of gt: the slot stays; of eq: it lies on the cut
  auto sort_out = [&](int from, uint32_t& gt, uint32_t& eq) {
    gt = eq = 0;
#pragma unroll
    for (int k = 0; k < kTimes; ++k)
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = from + (k * kThreads + tid) * kEach + j;
        const uint32_t w = key_of(x[k][j]);
        const bool end = i < lo || i >= hi;
        if (i < s1 && (end || (want > 0 && w > key)))
          gt |= 1u << (k * kEach + j);
        if (i < s1 && !end && want > 0 && w == key)
          eq |= 1u << (k * kEach + j);
      }
  };
  int bg = 0, be = 0;            // such slots in the CTAs before
  if (C > 1) {
    int ng = 0, ne = 0;
#pragma unroll 1
    for (int from = s0; from < s1; from += kHeld) {
      if (!held) load(from);
      uint32_t gt, eq;
      sort_out(from, gt, eq);
      ng += __popc(gt);
      ne += __popc(eq);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ng += __shfl_xor_sync(0xffffffffu, ng, o);
      ne += __shfl_xor_sync(0xffffffffu, ne, o);
    }
    if (lane == 0) {
      sh.warp_n[0][warp] = ng;
      sh.warp_n[1][warp] = ne;
    }
    __syncthreads();
    if (tid < C) {               // to every CTA
      int g = 0, e = 0;
      for (int w = 0; w < kWarps; ++w) {
        g += sh.warp_n[0][w];
        e += sh.warp_n[1][w];
      }
      Shared<kWarps>* to = cluster.map_shared_rank(&sh, tid);
      to->n_gt[me] = g;
      to->n_eq[me] = e;
    }
    cluster.sync();
    for (int r = 0; r < me; ++r) {
      bg += sh.n_gt[r];
      be += sh.n_eq[r];
    }
  }
#pragma unroll 1
  for (int from = s0; from < s1; from += kHeld) {
    if (!held) load(from);
    uint32_t gt, eq;
    sort_out(from, gt, eq);
#pragma unroll
    for (int k = 0; k < kTimes; ++k) {
      if (from + k * kThreads * kEach >= s1) break;   // (uniform)
      const uint32_t g = gt >> (k * kEach) & ((1 << kEach) - 1);
      const uint32_t e = eq >> (k * kEach) & ((1 << kEach) - 1);
      const int ng = __popc(g), ne = __popc(e);
      int rg = ng, re = ne;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int vg = __shfl_up_sync(0xffffffffu, rg, o);
        const int ve = __shfl_up_sync(0xffffffffu, re, o);
        if (lane >= o) {
          rg += vg;
          re += ve;
        }
      }
      __syncthreads();           // (the last turn's sums have been read)
      if (lane == 31) {
        sh.warp_n[0][warp] = rg;
        sh.warp_n[1][warp] = re;
      }
      __syncthreads();
      int vg = lane < kWarps ? sh.warp_n[0][lane] : 0;
      int ve = lane < kWarps ? sh.warp_n[1][lane] : 0;
      int tg = vg, te = ve;      // of all warps, of those before
      vg = lane < warp ? vg : 0;
      ve = lane < warp ? ve : 0;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        tg += __shfl_xor_sync(0xffffffffu, tg, o);
        te += __shfl_xor_sync(0xffffffffu, te, o);
        vg += __shfl_xor_sync(0xffffffffu, vg, o);
        ve += __shfl_xor_sync(0xffffffffu, ve, o);
      }
      int eq_before = be + ve + re - ne;       // slots on the cut before mine
      int at = bg + vg + rg - ng + min(eq_before, left);
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        bool keep = g >> j & 1;
        if (e >> j & 1) {
          keep = eq_before < left;
          ++eq_before;
        }
        if (keep) {
          kept[at] = from + (k * kThreads + tid) * kEach + j;
          if (mass_out) mass_out[at] = x[k][j];
          ++at;
        }
      }
      bg += tg;
      be += te;
    }
  }
  // ---- the codes
  // -----------------------------------------------------------------
  if (C > 1) cluster.sync(); else __syncthreads();  // the list is there
  const int page_bits = __ffs(a.page) - 1;
  const int pages = (a.budget + a.page - 1) >> page_bits;
  // kept[j] >= j grows with j: the first pages stay, as long as their last slot
  // does
  if (tid == 0) sh.stay = 0;
  __syncthreads();
  for (int p = tid; p < pages; p += kThreads) {
    const int last = min((p + 1) << page_bits, a.budget) - 1;
    if (kept[last] != last) break;           // (so of all after it)
    atomicMax(&sh.stay, p + 1);
  }
  __syncthreads();
  constexpr int kItems = kWarps / kOf, kOfThreads = 32 * kOf;
  const int slot = tid / kOfThreads, t = tid % kOfThreads;
  const int per_slot = a.D / 16;             // units of a slot
  // u / per_slot for the units of a page, u < 2048, exactly
  const uint32_t by = (65536 + per_slot - 1) / per_slot;
  const int* table = a.table + (long long)b * a.max_pages;
  const int round = C * kItems;              // pages
  // kept slots of this thread's units of page p (-1: none) and their pages' ids
  int from[kUnits], ids[kUnits], id = -1;
  auto look = [&](int p) {
    const int base = p << page_bits;
    const int units =
        p < pages ? (min(a.budget - base, a.page)) * per_slot : 0;
    if (p < pages) id = table[p];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int u = t + k * kOfThreads;
      from[k] = u < units ? kept[base + (int)(u * by >> 16)] : -1;
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
      ids[k] = from[k] >= 0 ? table[from[k] >> page_bits] : 0;
  };
  const int first = sh.stay + me * kItems + slot;
  look(first);
#pragma unroll 1
  for (int p0 = sh.stay; p0 < pages; p0 += round) {
    const int p = p0 + me * kItems + slot;
    const int to_id = id;
    uint4 w[2][kUnits];
    uint32_t e[kUnits];                      // the scales' exponents, k and v
    uint32_t live = 0;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      w[0][k] = w[1][k] = make_uint4(0, 0, 0, 0);
      e[k] = 127 | 127 << 8;
      if (from[k] < 0) continue;
      const int u = t + k * kOfThreads;
      live |= 1u << k;
      if (ids[k] < 0 || ids[k] >= a.num_pages) {  // such a page counts as zeros
        raise_error(a.err, kErrBadIndex);
        continue;
      }
      const long long ph = (long long)ids[k] * a.Hkv + h;
      const long long of =
          (ph * a.page + (from[k] & (a.page - 1))) * a.D +
          (u - (int)(u * by >> 16) * per_slot) * 16;
      w[0][k] = *reinterpret_cast<const uint4*>(a.codes[0] + of);
      w[1][k] = *reinterpret_cast<const uint4*>(a.codes[1] + of);
      e[k] = (__float_as_uint(a.scale[0][ph]) >> 23 & 255) |
             (__float_as_uint(a.scale[1][ph]) >> 23 & 255) << 8;
    }
    look(p + round);                         // (lists and ids do not change)
    int top[2] = {kMinExp, kMinExp};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        // (a NaN as the largest code)
        const uint32_t c = min(largest(w[kv][k]), 0x7eu);
        top[kv] = max(top[kv],
                      scale_exponent(c) + (int)(e[k] >> (8 * kv) & 255) - 127);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1)
        top[kv] = max(top[kv], __shfl_xor_sync(0xffffffffu, top[kv], o));
      if (lane == 0) sh.exp[kv][warp] = top[kv];
    }
    // All of the round's slots have been read before one is written, by any CTA
    // of the cluster: its barrier orders the reads before the writes.  (A
    // relaxed one takes 3 us less for the batch above, and only that every word
    // has its part in `top` would hold the writes back.  Arriving before the
    // maxima are taken: 122 us, but 20.4 and 251 to 259.)
    if (C > 1) cluster.sync(); else __syncthreads();
    // the next round's codes on their way to L2
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
      if (from[k] >= 0 && ids[k] >= 0 && ids[k] < a.num_pages) {
        const int u = t + k * kOfThreads;
        const long long of =
            (((long long)ids[k] * a.Hkv + h) * a.page +
             (from[k] & (a.page - 1))) * a.D +
            (u - (int)(u * by >> 16) * per_slot) * 16;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.codes[0] + of));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.codes[1] + of));
      }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        top[kv] = max(top[kv], sh.exp[kv][slot * kOf + i]);
      top[kv] = min(top[kv], 127);           // (a scale that is no number)
    }
    if (p < pages && to_id >= 0 && to_id < a.num_pages) {
      const long long ph = (long long)to_id * a.Hkv + h;
      const long long to = ph * a.page * a.D;
      if (t < 2)
        a.scale[t][ph] =
            __uint_as_float((uint32_t)((t ? top[1] : top[0]) + 127) << 23);
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        if (!(live >> k & 1)) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          uint4& c4 = w[kv][k];
          const int off = (int)(e[k] >> (8 * kv) & 255) - 127 - top[kv];
          if (off != 0) {
            c4.x = requant4(c4.x, off);
            c4.y = requant4(c4.y, off);
            c4.z = requant4(c4.z, off);
            c4.w = requant4(c4.w, off);
          }
          *reinterpret_cast<uint4*>(a.codes[kv] + to +
                                    (long long)(t + k * kOfThreads) * 16) = c4;
        }
      }
    } else if (p < pages && t == 0) {
      raise_error(a.err, kErrBadIndex);
    }
    __syncthreads();                         // (the exponents have been read)
  }
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool evict_sizes_ok(int B, int Hkv, int page, int budget) {
  return B >= 1 && Hkv >= 1 && Hkv <= 4096 && B <= (1 << 20) &&
         (long long)B * Hkv * kMaxCluster <= 0x7fffffffll &&
         (page == 16 || page == 32 || page == 64 || page == 128) &&
         budget >= 1 && budget <= (1 << 30);
}

template <int kThreads, int kOf, int kUnits>
cudaError_t launch(const EvictArgs& a, int C, cudaStream_t s) {
  PdlLaunch L(dim3((unsigned)(a.B * a.Hkv * C)), dim3(kThreads), 0, s, C);
  return cudaLaunchKernelEx(&L.cfg, kv_evict_kernel<kThreads, kOf, kUnits>, a);
}
template <int kThreads>
cudaError_t launch_units(const EvictArgs& a, int C, cudaStream_t s) {
  const int units = a.page * a.D / 16;       // of a page, up to 2048
  return units <= 128    ? launch<kThreads, 1, 4>(a, C, s)
         : units <= 256  ? launch<kThreads, 2, 4>(a, C, s)
         : units <= 512  ? launch<kThreads, 4, 4>(a, C, s)
         : units <= 1024 ? launch<kThreads, 8, 4>(a, C, s)
                         : launch<256, 8, 8>(a, C, s);
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_kv_evict_workspace_bytes(int B, int Hkv, int page, int budget) {
  using namespace dflash;
  if (!evict_sizes_ok(B, Hkv, page, budget)) return 0;
  const size_t need = (size_t)B * Hkv * budget * sizeof(int);  // the kept slots
  return (need + 255) & ~(size_t)255;
}

dflash_status dflash_kv_evict(
    const float* mass, int64_t ld_mass, uint8_t* k_codes, uint8_t* v_codes,
    float* k_scale, float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, int B, int Hkv, int D, int page, int num_pages,
    int max_pages, int budget, int sink, int recent, float* mass_out,
    int64_t ld_out, int32_t* new_len, int32_t* kept, void* ws,
    size_t ws_bytes, dflash_stream_t stream) {
  using namespace dflash;
  if (!(mass && k_codes && v_codes && k_scale && v_scale && page_table &&
        kv_len && new_len && ws) || new_len == kv_len || mass_out == mass)
    return DFLASH_ERR_INVALID_ARG;
  if (!cache_sizes_ok(B, 1, Hkv, Hkv, D, page, num_pages, max_pages) ||
      !evict_sizes_ok(B, Hkv, page, budget))
    return DFLASH_ERR_INVALID_ARG;
  if (sink < 0 || recent < 0 || (long long)sink + recent > budget ||
      ld_mass < 1 || (mass_out && ld_out < 1))
    return DFLASH_ERR_INVALID_ARG;
  if (!aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) ||
      !aligned_to(ws, 256) ||
      ws_bytes < dflash_kv_evict_workspace_bytes(B, Hkv, page, budget))
    return DFLASH_ERR_INVALID_ARG;
  // slots of the new lengths' weights
  const long long most =
      std::min<long long>(std::min<long long>(budget, ld_mass),
                          (long long)max_pages * page);
  if (mass_out && ld_out < most) return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  EvictArgs a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.mass = mass;
  a.ld_mass = ld_mass;
  a.ld_out = ld_out;
  a.codes[0] = k_codes;
  a.codes[1] = v_codes;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.table = page_table;
  a.kv_len = kv_len;
  a.B = B;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.budget = budget;
  a.sink = sink;
  a.recent = recent;
  a.mass_out = mass_out;
  a.new_len = new_len;
  a.kept = kept ? kept : static_cast<int*>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // CTAs to a head: as many as make four small ones to an SM, half of the
  // sequences being shorter than their budget, if there are slots for them;
  // large ones where the heads leave most SMs without any.
  const long long slots =
      std::min<long long>(ld_mass, (long long)max_pages * page);
  int C = 1;
  while (C < kMaxCluster && (long long)B * Hkv * C * 2 <= 8ll * sms &&
         slots > 256ll * C)
    C *= 2;
  const bool few = (long long)B * Hkv * C <= sms;
  const cudaError_t e =
      few ? launch_units<512>(a, C, s) : launch_units<256>(a, C, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
