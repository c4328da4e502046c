// Log probabilities of given tokens, their ranks, the rows' entropies and
// their most likely tokens.
//
// Mathematics, in bits: with c = log2(e) / T and a whole number r near the
// largest l c, y = l c - r (one rounding), w = 2^y, S = sum w, U = sum w y:
//   lse = ln2 (r + log2 S);   ln p_v = ln2 (y_v - log2 S);
//   entropy = ln2 (log2 S - U / S).
// One pass keeps r (at first of the given token's l c), S and U of what a thread
// has seen; when r grows by h, U becomes 2^-h (U - h S) and S 2^-h S, and two
// threads' sums join likewise.  A token's rank is the number of tokens before it in
// the order (logit descending, id ascending), so its logit is fetched first and
// the pass counts: words before the token those above the next smaller number,
// words after it those above its logit.
//
// The K most likely: the K-th largest maximum of 64 groups of threads bounds the
// K-th largest logit of the slice from below.  Of the threads that reach it most
// do so with the words of their maximum alone, which they read again; the others
// have their whole part read again, from L2, a warp at a time for each. The few
// more than K candidates are ranked by counting.  A cluster of CTAs owns a row;
// the first of them joins the CTAs' sums and lists.  What overflows the list
// (ties by the thousand, or a row masked by the type's lowest value whose other
// tokens lie in fewer than K groups: 288 such rows 1140 us, masked by -inf 55)
// is found by K searches for the next largest instead.
//
// What bounds it: in batches instructions (25 a logit, 70 % of the issue slots)
// and the steps at a row's end; for one row the chain of steps.  288 rows of
// 151936 fp32 logits 45 us with 20 alternatives, 35 us without (4.9 TB/s), bf16
// 38 us, one bf16 row 5.9 us.  (Words on their way through shared memory, four
// to twelve of a thread in flight instead of two: 49 to 51 us.)
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
constexpr int kGroups = 64;     // of threads, for the bound of the top K
constexpr int kGroupOf = kThreads / kGroups;
constexpr int kMost = DFLASH_MAX_ALTERNATIVES;
constexpr int kList = 1024;     // candidates of a CTA
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
static_assert(kMost <= kGroups, "");

struct Args {
  const void* logits;
  long long ld;
  const float* temperature;
  const int* token;
  int R, V, K, slice;   // slice: tokens per CTA
  float *logprob, *lse, *entropy, *top;
  int *rank, *top_id;
  int* err;
};

// m: largest logit; r: the reference, -inf while there is none; s, u: the sums.
struct Sums {
  float m, r, s, u;
};
// Products l c from this size on are rounded by whole bits, and more: there y is
// what their rounded values differ by, never above 0.
constexpr float kFar = 0x1p30f;
constexpr float kLowest = -0x1.fffffep127f;  // instead of a finite l's -inf
__device__ __forceinline__ float far_bits(float l, float c, float ref) {
  return l == -INFINITY
             ? -INFINITY
             : fminf(fmaxf(__fmul_rn(l, c), kLowest) + ref, 0.f);
}
// 2^h u and s of a reference that is h higher.
__device__ __forceinline__ void lower(float h, float& s, float& u) {
  h = fmaxf(h, -1024.f);             // (the same 0, and no infinite h s)
  const float f = tc::ex2_approx(h);
  u = f * fmaf(h, s, u);
  s *= f;
}
__device__ __forceinline__ Sums join(Sums a, Sums b) {
  if (b.r > a.r) {
    const Sums t = a;
    a = b;
    b = t;
  }
  a.m = fmaxf(a.m, b.m);
  const float h = b.r - a.r;         // (no reference, an infinite one: -inf, NaN)
  if (h > -INFINITY) {
    lower(h, b.s, b.u);
    a.s += b.s;
    a.u += b.u;
  }
  return a;
}

// What the CTAs of a row hand to the first of them.
struct Shared {
  Sums sums[kMaxCluster];
  int before[kMaxCluster];
  int odd[kMaxCluster];
  u64 top[kMaxCluster][kMost];
  int n_top[kMaxCluster];
  // this CTA's own
  Sums warp_sums[kWarps];
  int warp_before[kWarps], warp_odd[kWarps];
  float group_max[kGroups];
  float bound;
  int listed;
  u64 list[kList];
  u64 warp_best[kWarps];
};

// Order-preserving key of a logit that is no NaN (equal for -0 and 0).
__device__ __forceinline__ u64 word_of(float x, int id) {
  const uint32_t w = __float_as_uint(x + 0.f);
  return (u64)(w & 0x80000000u ? ~w : w | 0x80000000u) << 32 | (uint32_t)~id;
}
__device__ __forceinline__ float value_of(u64 word) {
  const uint32_t k = (uint32_t)(word >> 32);
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A 16-byte word of logits, as fp32.
template <typename T>
struct Words {
  static constexpr int N = 16 / sizeof(T);
  __device__ static __forceinline__ void get(const uint4& w, float (&f)[N]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(x[i] << 16);
        f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
      }
    }
  }
};

// max of three numbers; a NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The next smaller number (of -inf: a NaN, above which nothing is).
__device__ __forceinline__ float next_below(float x) {
  const int w = __float_as_int(x);
  return x == 0.f ? __int_as_float(0x80000001)
                  : __int_as_float(x > 0.f ? w - 1 : w + 1);
}
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <typename T, bool kTop, bool kRank>
__global__ void __launch_bounds__(kThreads, 2)
    logprobs_kernel(const __grid_constant__ Args a) {
  constexpr int N = Words<T>::N;
  constexpr int kAhead = 2;          // words in flight
  extern __shared__ uint4 smem16[];
  Shared& sh = *reinterpret_cast<Shared*>(smem16);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_trigger();
  pdl_wait();
  const int r = blockIdx.x / C;
  const T* row = static_cast<const T*>(a.logits) + (long long)r * a.ld;
  auto temperature = [&](bool& odd) {
    const float t = a.temperature ? a.temperature[r] : 1.f;
    odd = !(t >= 0x1p-126f && t < INFINITY);
    return odd ? 1.f : t;
  };
  bool odd;
  const float c = kLog2e / temperature(odd);
  const int token = a.token ? a.token[r] : -1;
  const bool given = token >= 0 && token < a.V;
  const float mine = given ? to_f32(row[token]) : 0.f;

  // Words of 16 bytes that start on a 16-byte boundary: word i holds tokens
  // i N - skew .. of the row.  This CTA's are [w0, w1).
  const int skew = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const T* base = row - skew;
  const int words = (int)(((long long)a.V + skew + N - 1) / N);
  const int per = a.slice / N;
  const int w0 = min(words, me * per), w1 = min(words, w0 + per);
  // whole words only; the others are read by token
  const int full0 = skew ? 1 : 0, full1 = (int)(((long long)a.V + skew) / N);
  auto whole = [&](int i) { return i >= full0 && i < full1; };
  auto fetch = [&](int i) {
    uint4 w;
    if (whole(i)) {
      w = __ldg(reinterpret_cast<const uint4*>(base) + i);
    } else {                       // the row's ends, filled up with -inf
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          const long long v = (long long)i * 4 + j - skew;
          x[j] = v >= 0 && v < a.V
                     ? reinterpret_cast<const uint32_t*>(row)[v] : 0xff800000u;
        } else {
          x[j] = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const long long v = (long long)i * 8 + 2 * j + h - skew;
            x[j] |= (uint32_t)(v >= 0 && v < a.V
                                   ? reinterpret_cast<const uint16_t*>(row)[v]
                                   : 0xff80u)
                    << (16 * h);
          }
        }
      }
      w = make_uint4(x[0], x[1], x[2], x[3]);
    }
    return w;
  };

  Sums acc{-INFINITY, -INFINITY, 0.f, 0.f};
  // The given token's logit is a good first reference: none is too high that
  // some logit has.  (It is often the largest, and no thread raises it then.)
  if (given && fabsf(mine * c) < INFINITY) acc.r = ceilf(mine * c);
  const int token_at =               // its word
      given ? (int)(((long long)token + skew) / N) : -1;
  int before = 0;
  int best = 0;                      // the first word of those with the maximum
  float others = -INFINITY;          // the largest of all other words
  const float below = next_below(mine);
  const uint64_t c2 = pack2(c, c);
  auto take = [&](const uint4 (&raw)[kAhead], int first, int n) {
    float f[kAhead][N];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k >= n) break;
      Words<T>::get(raw[k], f[k]);
#pragma unroll
      for (int j = 0; j < N; j += 2) top = max_nan(top, f[k][j], f[k][j + 1]);
    }
    if (top != top) {                // a NaN: left out
      odd = true;
      top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (f[k][j] != f[k][j]) f[k][j] = -INFINITY;
          top = fmaxf(top, f[k][j]);
        }
      }
    }
    if (kTop) {
      others = fmaxf(others, fminf(top, acc.m));
      best = top > acc.m ? first : best;
    }
    acc.m = fmaxf(acc.m, top);
    const float bits = fmaxf(top * c, kLowest);
    if (bits > acc.r) {
      const float r = ceilf(bits);
      // (a step of -inf, at first, before +inf or where it passes fp32's range,
      // leaves nothing)
      lower(acc.r - r, acc.s, acc.u);
      acc.r = r;
    }
    // (far: NaNs, which are seen below)
    const float ref =
        fabsf(acc.r) < kFar ? -acc.r : __int_as_float(0x7fffffff);
    const uint64_t ref2 = pack2(ref, ref);
    uint64_t s2 = 0, u2 = 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k >= n) break;
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        const uint64_t y = fma2(pack2(f[k][j], f[k][j + 1]), c2, ref2);
        float y0, y1;
        unpack2(y, y0, y1);
        const uint64_t w = pack2(tc::ex2_approx(y0), tc::ex2_approx(y1));
        s2 = add2(s2, w);
        u2 = fma2(w, y, u2);
      }
    }
    float s0, s1, u0, u1;
    unpack2(s2, s0, s1);
    unpack2(u2, u0, u1);
    u0 += u1;
    if (u0 != u0) {                  // far, or -inf, whose weight is 0: again
      s0 = s1 = u0 = 0.f;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float y = ref == ref ? fmaf(f[k][j], c, ref)
                                     : far_bits(f[k][j], c, -acc.r);
          const float w = tc::ex2_approx(y);
          s0 += w;
          if (y > -INFINITY) u0 = fmaf(w, y, u0);
        }
      }
    }
    acc.s += s0 + s1;
    acc.u += u0;
    if constexpr (kRank) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (k >= n) break;
        const int word = first + k * kThreads;
        if (word == token_at || mine == -INFINITY) {
          const long long at = (long long)word * N - skew;
#pragma unroll
          for (int j = 0; j < N; ++j)
            before += f[k][j] > mine ||
                      (f[k][j] == mine && at + j < token && at + j >= 0);
        } else {
          const float than = word < token_at ? below : mine;
#pragma unroll
          for (int j = 0; j < N; ++j) before += f[k][j] > than;
        }
      }
    }
  };
  {
    uint4 raw[kAhead], next[kAhead];
    auto ask = [&](int i, uint4 (&to)[kAhead]) {
      const int n = min(kAhead, (w1 - i + kThreads - 1) / kThreads);
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < n) to[k] = fetch(i + k * kThreads);
      return n;
    };
    int i = w0 + tid, n = ask(i, raw);
#pragma unroll 1
    while (n > 0) {
      const int n2 = ask(i + kAhead * kThreads, next);
      take(raw, i, n);
      i += kAhead * kThreads;
      n = n2;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) raw[k] = next[k];
    }
  }

  // ---- the CTA's sums ------------------------------------------------------
  const float my_max = acc.m;
  auto fold = [&](Sums& x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Sums y{__shfl_xor_sync(0xffffffffu, x.m, o),
                   __shfl_xor_sync(0xffffffffu, x.r, o),
                   __shfl_xor_sync(0xffffffffu, x.s, o),
                   __shfl_xor_sync(0xffffffffu, x.u, o)};
      x = join(x, y);                // (both lanes get the same bits)
    }
  };
  fold(acc);
  if (kRank) before = __reduce_add_sync(0xffffffffu, before);
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) {
    sh.warp_sums[warp] = acc;
    sh.warp_before[warp] = before;
    sh.warp_odd[warp] = odd;
  }
  if (kTop) {
    float g = my_max;
#pragma unroll
    for (int o = kGroupOf / 2; o; o >>= 1)
      g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid % kGroupOf == 0) sh.group_max[tid / kGroupOf] = g;
    if (tid == 0) sh.listed = 0;
  }
  __syncthreads();
  Shared* first = cluster.map_shared_rank(&sh, 0);
  if (tid < 32) {
    Sums x = tid < kWarps ? sh.warp_sums[tid]
                          : Sums{-INFINITY, -INFINITY, 0.f, 0.f};
    fold(x);
    const int b =
        __reduce_add_sync(0xffffffffu, tid < kWarps ? sh.warp_before[tid] : 0);
    const int o =
        __reduce_or_sync(0xffffffffu, tid < kWarps ? sh.warp_odd[tid] : 0);
    // every CTA of the cluster has started
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (tid == 0) {
      first->sums[me] = x;
      first->before[me] = b;
      first->odd[me] = o;
    }
  } else {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }

  // ---- the CTA's K most likely
  // ------------------------------------------------
  if (kTop) {
    if (tid < kGroups) {             // the K-th largest maximum
      const float g = sh.group_max[tid];
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < kGroups; ++i) {
        const float x = sh.group_max[i];
        above += x > g || (x == g && i < tid);
      }
      if (above == a.K - 1) sh.bound = g;
    }
    __syncthreads();
    const float bound = sh.bound;
    // (-inf: fewer than K groups hold any token; then every token above it is a
    // candidate)
    auto offer = [&](int i) {
      float f[N];
      Words<T>::get(fetch(i), f);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (f[j] >= bound && f[j] > -INFINITY) {
          const int to = atomicAdd(&sh.listed, 1);
          if (to < kList)
            sh.list[to] = word_of(f[j], (int)((long long)i * N + j - skew));
        }
    };
    const bool reaches = my_max >= bound && my_max > -INFINITY;
    const bool again = reaches && others >= bound;
    if (reaches && !again) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (best + k * kThreads < w1) offer(best + k * kThreads);
    }
    uint32_t reach = __ballot_sync(0xffffffffu, again);
    while (reach) {                  // the whole warp reads one thread's part
      const int who = __ffs(reach) - 1;
      reach &= reach - 1;
#pragma unroll 2
      for (int i = w0 + warp * 32 + who + lane * kThreads; i < w1;
           i += 32 * kThreads)
        offer(i);
    }
    __syncthreads();
    int n = sh.listed;
    if (n <= kList) {
      for (int i = tid; i < n; i += kThreads) {
        const u64 x = sh.list[i];
        int above = 0;
        for (int j = 0; j < n; ++j) above += sh.list[j] > x;
        if (above < a.K) first->top[me][above] = x;
      }
      n = min(n, a.K);
    } else {                         // the next largest, K times
      u64 last = ~0ull;
      n = a.K;                       // there are more than kList
      for (int k = 0; k < a.K; ++k) {
        u64 best = 0;
        for (int i = w0 + tid; i < w1; i += kThreads) {
          float f[N];
          Words<T>::get(fetch(i), f);
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (f[j] > -INFINITY) {
              const u64 x = word_of(f[j], (int)((long long)i * N + j - skew));
              if (x < last && x > best) best = x;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
          best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0) sh.warp_best[warp] = best;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) best = max(best, sh.warp_best[i]);
        __syncthreads();
        last = best;
        if (tid == 0) first->top[me][k] = best;
      }
    }
    if (tid == 0) first->n_top[me] = n;
  }
  cluster.sync();
  if (me != 0) return;

  // ---- the row
  // -----------------------------------------------------------------
  Sums x{-INFINITY, -INFINITY, 0.f, 0.f};
  int rank = 0, any_odd = 0;
  for (int i = 0; i < C; ++i) {
    x = join(x, sh.sums[i]);
    rank += sh.before[i];
    any_odd |= sh.odd[i];
  }
  // (an x beyond fp32's range counts as infinite)
  const bool empty = x.m == -INFINITY;
  const bool infinite = !empty && !(fabsf(x.r) < INFINITY);
  const bool far = fabsf(x.r) >= kFar;
  const float log_s = log2f(x.s);
  const float nan = __int_as_float(0x7fffffff);
  // (read again: held over the pass it cost the registers of something else)
  bool known;
  const float t = temperature(known);
  const float lse = empty      ? -INFINITY
                    : infinite ? x.r
                    : far      ? x.m / t + log_s * kLn2
                               : (x.r + log_s) * kLn2;
  // (ln p in one rounding of y: exact for the row's likeliest tokens)
  auto log_p = [&](float l) {
    if (far) return (far_bits(l, c, -x.r) - log_s) * kLn2;
    const float y = fmaf(l, c, -x.r);
    return y < -kFar ? l / t - lse : (y - log_s) * kLn2;
  };
  if (tid == 0) {
    if (any_odd || empty || infinite) raise_error(a.err, kErrNonfinite);
    if (token >= a.V || token < -1) raise_error(a.err, kErrBadIndex);
    if (a.lse) a.lse[r] = lse;
    if (a.entropy)
      a.entropy[r] = empty || infinite
                         ? nan
                         : fmaxf((log_s - x.u / x.s) * kLn2, 0.f);
    if (a.logprob)
      a.logprob[r] = token == -1                   ? 0.f
                     : !given || empty || infinite ? nan
                                                   : log_p(mine);
    if (kRank) a.rank[r] = given && mine == mine ? rank : -1;
  }
  if (kTop) {
    const int lists = C * kMost;
    for (int i = tid; i < a.K; i += kThreads) {
      a.top[(long long)r * a.K + i] = -INFINITY;
      a.top_id[(long long)r * a.K + i] = -1;
    }
    __syncthreads();
    for (int i = tid; i < lists; i += kThreads) {
      const int from = i / kMost, k = i % kMost;
      if (k >= sh.n_top[from]) continue;
      const u64 w = sh.top[from][k];
      int above = k;                 // its own list is sorted
      for (int j = 0; j < C; ++j)
        if (j != from)
          for (int q = 0; q < sh.n_top[j] && above < a.K; ++q) {
            if (sh.top[j][q] < w) break;
            ++above;
          }
      if (above < a.K) {
        const float v = value_of(w);
        a.top[(long long)r * a.K + above] =
            infinite ? nan : log_p(v);
        a.top_id[(long long)r * a.K + above] = (int)~(uint32_t)w;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const Args& args, int sms, cudaStream_t s) {
  Args a = args;
  // CTAs of a row: as many as all rows' find room at once, two to an SM (the
  // chain of steps at a CTA's end is then paid once: 288 rows of 151936 fp32
  // logits, at an earlier step, 51 us, with two CTAs each 55), with 4096 tokens
  // each
  int C = 1;
  while (C < kMaxCluster && (long long)a.R * C <= sms && a.V > 4096 * C)
    C *= 2;
  const int N = 16 / sizeof(T);
  // (a row may start anywhere in its first word)
  const long long words = ((long long)a.V + 2 * N - 2) / N;
  a.slice = (int)((words + C - 1) / C * N);
  if ((long long)a.R * C > 0x7fffffffll) return cudaErrorNotSupported;
  const bool top = a.K > 0, rank = a.rank != nullptr;
  auto* f = top ? rank ? logprobs_kernel<T, true, true>
                       : logprobs_kernel<T, true, false>
            : rank ? logprobs_kernel<T, false, true>
                   : logprobs_kernel<T, false, false>;
  PdlLaunch L(dim3((unsigned)(a.R * C)), dim3(kThreads), sizeof(Shared), s, C);
  return cudaLaunchKernelEx(&L.cfg, f, a);
}
static_assert(sizeof(Shared) <= 48 * 1024, "");

}  // namespace
}  // namespace dflash

extern "C" dflash_status dflash_logprobs(
    const void* logits, int64_t ld, dflash_dtype dt, const float* temperature,
    const int32_t* token, int R, int V, int K, float* logprob, int32_t* rank,
    float* lse, float* entropy, float* top, int32_t* top_id,
    dflash_stream_t stream) {
  using namespace dflash;
  if (!logits || (dt != DFLASH_BF16 && dt != DFLASH_FP32))
    return DFLASH_ERR_INVALID_ARG;
  if (R < 1 || V < 1 || V > 0x7fffff00 || ld < V || K < 0 || K > kMost)
    return DFLASH_ERR_INVALID_ARG;
  if ((logprob || rank) && !token) return DFLASH_ERR_INVALID_ARG;
  if ((K > 0) != (top != nullptr) || (K > 0) != (top_id != nullptr))
    return DFLASH_ERR_INVALID_ARG;
  const uintptr_t size = dt == DFLASH_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(logits) % size)
    return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  Args a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.logits = logits;
  a.ld = ld;
  a.temperature = temperature;
  a.token = token;
  a.R = R;
  a.V = V;
  a.K = K;
  a.logprob = logprob;
  a.lse = lse;
  a.entropy = entropy;
  a.top = top;
  a.rank = rank;
  a.top_id = top_id;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == DFLASH_FP32 ? launch<float>(a, sms, s)
                                          : launch<__nv_bfloat16>(a, sms, s);
  return e == cudaSuccess            ? DFLASH_OK
         : e == cudaErrorNotSupported ? DFLASH_ERR_UNSUPPORTED
                                      : DFLASH_ERR_CUDA;
}
