// Eviction from the paged 8-bit cache by the attention weight that tokens have
// gathered.
//
// Mathematics.  Of a key head's n > budget slots the first `sink` and the last
// `recent` stay, and of the others the budget - sink - recent of largest weight
// (ties: the lower slot).  That is a cut in the order of 32-bit keys, found by
// three histograms (11, 11 and 10 bits), and the first few of the slots that lie
// on it.  The kept slots move to slots 0 .. budget - 1 in their order.  A page
// that gets other tokens gets a scale of its own, the least power of two with
// max |x| <= 448 s, as an append would give it: codes move exactly but for those
// that become subnormal.
//
// Two launches.  The first has one CTA per sequence and key head: the cut, the
// list of kept slots, their weights.  The second moves codes, a CTA for each
// (new page, key head, k or v).  It moves in place: slots only move down, so a
// page may be written once every lower page that takes a slot of it has read
// that.  A CTA takes its number from a counter, lower pages first, reads its
// slots into registers, says so with a flag, and only then waits for the flags
// of those few pages, whose CTAs have all started and wait for nothing before
// their flags: the waits end.
#include <cuda_fp8.h>

#include <algorithm>

#include "kernels.h"
#include "tc_ptx.cuh"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

constexpr int kMinExp = -64;      // smallest exponent of a block scale
constexpr int kSelect = 1024;     // threads of a selecting CTA
constexpr int kMove = 128;        // of a moving one
constexpr int kBins = 2048;
constexpr int kEach = 4;          // slots a thread takes at a time

struct EvictArgs {
  const float* mass;
  long long ld_mass, ld_out;      // slots of a head in mass and mass_out
  uint8_t* codes[2];
  float* scale[2];
  const int *table, *kv_len;
  int B, Hkv, D, page, num_pages, max_pages, budget, sink, recent;
  float* mass_out;                // may be NULL
  int *new_len, *kept;
  int pages;                      // new pages of a sequence, at most
  unsigned* flags;                // [pages][B][Hkv][2]: read
  unsigned* ticket;
  int* err;
  uint64_t wait_ns;
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

__global__ void __launch_bounds__(kSelect, 1)
    kv_evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ int warp_n[2][32];
  __shared__ int s_bin, s_left, s_gt, s_eq;
  pdl_trigger();
  pdl_wait();
  const int h = blockIdx.x % a.Hkv, b = blockIdx.x / a.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * a.Hkv + h;
  // the flags of this head's new pages, and the counter
  for (int i = tid; i < a.pages * 2; i += kSelect)
    a.flags[((long long)(i >> 1) * a.B * a.Hkv + bh) * 2 + (i & 1)] = 0;
  if (blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  bool bad = false;
  const int n = length_of(a, b, &bad);
  const float* mass = a.mass + bh * a.ld_mass;
  int* kept = a.kept + bh * a.budget;
  if (h == 0 && tid == 0) {
    a.new_len[b] = min(n, a.budget);
    if (bad) raise_error(a.err, kErrBadIndex);
  }
  if (n <= a.budget) {
    for (int i = tid; i < a.budget; i += kSelect) kept[i] = i < n ? i : -1;
    if (a.mass_out)
      for (int i = tid; i < n; i += kSelect)
        a.mass_out[bh * a.ld_out + i] = mass[i];
    return;
  }
  // (n > budget >= sink + recent: the two ends do not meet)
  const int lo = a.sink, hi = n - a.recent;
  const int want = a.budget - a.sink - a.recent;
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
      for (int i = tid; i < kBins; i += kSelect) hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelect) {
        const float x = mass[i];
        const uint32_t k = key_of(x);
        nan |= x != x;
        if (pass == 0 || (k >> (shift + bits)) == prefix)
          atomicAdd(&hist[(k >> shift) & ((1 << bits) - 1)], 1);
      }
      __syncthreads();
      // the bin, counted from the largest, in which the left-th slot lies: a
      // thread has two bins, the largest ones first
      const int nb = 1 << bits;
      const int b1 = nb - 1 - 2 * tid, b0 = b1 - 1;
      const int c1 = b1 >= 0 ? hist[b1] : 0, c0 = b0 >= 0 ? hist[b0] : 0;
      int run = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      if (lane == 31) warp_n[0][warp] = run;
      __syncthreads();
      for (int w = 0; w < warp; ++w) run += warp_n[0][w];
      const int above = run - c0 - c1;       // slots in larger bins
      if (above < left && left <= run) {
        const bool in1 = left <= above + c1;
        s_bin = in1 ? b1 : b0;
        s_left = left - above - (in1 ? 0 : c1);
      }
      __syncthreads();
      prefix = prefix << bits | (uint32_t)s_bin;
      left = s_left;
      __syncthreads();
    }
    key = prefix;
    if (nan) raise_error(a.err, kErrNonfinite);
  }
  // ---- the kept slots in their order ---------------------------------------
  if (tid == 0) {
    s_gt = 0;
    s_eq = 0;
  }
  __syncthreads();
  for (int base = 0; base < n; base += kSelect * kEach) {
    const int i0 = base + tid * kEach;
    uint32_t gt = 0, eq = 0;
    float x[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = i0 + j;
      x[j] = i < n ? mass[i] : 0.f;
      if (i < n) {
        if (i < lo || i >= hi) {
          gt |= 1u << j;
        } else {
          const uint32_t k = key_of(x[j]);
          if (want > 0 && k > key) gt |= 1u << j;
          if (want > 0 && k == key) eq |= 1u << j;
        }
      }
    }
    int ng = __popc(gt), ne = __popc(eq);
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
    if (lane == 31) {
      warp_n[0][warp] = rg;
      warp_n[1][warp] = re;
    }
    __syncthreads();
    int bg = s_gt, be = s_eq, tg = 0, te = 0;
    for (int w = 0; w < kSelect / 32; ++w) {
      if (w < warp) {
        bg += warp_n[0][w];
        be += warp_n[1][w];
      }
      tg += warp_n[0][w];
      te += warp_n[1][w];
    }
    int eq_before = be + re - ne;            // slots on the cut before mine
    int at = bg + rg - ng + min(eq_before, left);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      bool keep = gt >> j & 1;
      if (eq >> j & 1) {
        keep = eq_before < left;
        ++eq_before;
      }
      if (keep) {
        kept[at] = i0 + j;
        if (a.mass_out) a.mass_out[bh * a.ld_out + at] = x[j];
        ++at;
      }
    }
    __syncthreads();
    if (tid == 0) {
      s_gt += tg;
      s_eq += te;
    }
    __syncthreads();
  }
}

// Exponent of the least power of two s with x <= 448 s (x a value of E4M3).
__device__ __forceinline__ int scale_exponent(float x) {
  const uint32_t w = __float_as_uint(x);
  if (w < 0x00800000u) return -1000;         // zero
  return (int)(w >> 23) - 127 - 8 + ((w & 0x7fffffu) > 0x600000u);
}
__device__ __forceinline__ uint32_t requant4(uint32_t w, float ratio) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const uint32_t c = __nv_cvt_float2_to_fp8x2(
        make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3);
    out |= c << (16 * i);
  }
  return out;
}

// A page of `page` slots of D codes is page * D / 16 units; kUnits of a thread.
template <int kUnits>
__global__ void __launch_bounds__(kMove)
    kv_evict_move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ unsigned s_item;
  __shared__ int s_exp[kMove / 32];
  __shared__ int s_late;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  if (tid == 0) {
    s_item = atomicAdd(a.ticket, 1u);
    s_late = 0;
  }
  __syncthreads();
  unsigned item = s_item;                    // (below the grid's 2^31)
  const int kv = item & 1;
  item >>= 1;
  const int h = item % a.Hkv;
  item /= a.Hkv;
  const int b = item % a.B, p = item / a.B;
  const long long bh = (long long)b * a.Hkv + h;
  bool bad = false;
  const int n = length_of(a, b, &bad);
  unsigned* flags = a.flags + bh * 2 + kv;
  const long long step = (long long)a.B * a.Hkv * 2;  // a page further
  const int s0 = p * a.page;
  const int s1 = min(min(n, a.budget), s0 + a.page);
  const int* kept = a.kept + bh * a.budget;
  // kept[j] >= j grows with j: the page stays if its last slot does
  if (n <= a.budget || s0 >= s1 || kept[s1 - 1] == s1 - 1) return;
  const int* table = a.table + (long long)b * a.max_pages;
  const int id = table[p];
  const int per = a.D / 16;                  // units of a slot
  const int units = (s1 - s0) * per;
  uint4 w[kUnits];
  int e[kUnits];                             // exponents of the units' scales
  int top = kMinExp;
  bool missing = id < 0 || id >= a.num_pages;
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int u = tid + k * kMove;
    w[k] = make_uint4(0, 0, 0, 0);
    e[k] = 0;
    if (u < units) {
      const int j = u / per;
      const int from = kept[s0 + j];
      const int fid = table[from / a.page];
      if (fid < 0 || fid >= a.num_pages) {   // such a page counts as zeros
        raise_error(a.err, kErrBadIndex);
      } else {
        const long long ph = (long long)fid * a.Hkv + h;
        w[k] = *reinterpret_cast<const uint4*>(
            a.codes[kv] + (ph * a.page + from % a.page) * a.D +
            (u - j * per) * 16);
        e[k] = (int)(__float_as_uint(a.scale[kv][ph]) >> 23) - 127;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const uint32_t m = __vmaxu4(
        __vmaxu4(w[k].x & 0x7f7f7f7fu, w[k].y & 0x7f7f7f7fu),
        __vmaxu4(w[k].z & 0x7f7f7f7fu, w[k].w & 0x7f7f7f7fu));
    const uint32_t c =
        min(max(max(m & 0xff, m >> 8 & 0xff), max(m >> 16 & 0xff, m >> 24)),
            0x7eu);                          // (a NaN as the largest code)
    const float x = __half2float(__half(
        __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
    top = max(top, scale_exponent(x) + e[k]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1)
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) s_exp[tid >> 5] = top;
  __syncthreads();                           // every slot has been read
  if (tid == 0) {
    __threadfence();
    asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(flags + p * step)
                 : "memory");
  }
  for (int i = 0; i < kMove / 32; ++i) top = max(top, s_exp[i]);
  top = min(top, 127);                       // (a scale that is no number)
  // ---- the lower pages that read this one ------------------------------------
  for (int d = p - 1 - tid; d >= 0; d -= kMove) {
    if (kept[(d + 1) * a.page - 1] < s0) break;
    const unsigned* f = flags + d * step;
    uint64_t t0 = 0;
    for (;;) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                   : "=r"(v)
                   : "l"(f)
                   : "memory");
      if (v) break;
      const uint64_t now = tc::globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > a.wait_ns) {
        s_late = 1;
        break;
      }
    }
  }
  __syncthreads();
  if (s_late || missing) {
    if (tid == 0) raise_error(a.err, s_late ? kErrTimeout : kErrBadIndex);
    return;
  }
  // ---- the page ------------------------------------------------------------------
  const long long ph = (long long)id * a.Hkv + h;
  uint8_t* dst = a.codes[kv] + ph * a.page * a.D;
  if (tid == 0)
    a.scale[kv][ph] = __uint_as_float((uint32_t)(top + 127) << 23);
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int u = tid + k * kMove;
    if (u >= units) continue;
    if (e[k] != top) {
      // below 2^-40 of the new scale a code is 0; above 2^40 they all are
      const float ratio = __uint_as_float(
          (uint32_t)(min(max(e[k] - top, -40), 40) + 127) << 23);
      w[k].x = requant4(w[k].x, ratio);
      w[k].y = requant4(w[k].y, ratio);
      w[k].z = requant4(w[k].z, ratio);
      w[k].w = requant4(w[k].w, ratio);
    }
    *reinterpret_cast<uint4*>(dst + (long long)u * 16) = w[k];
  }
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool evict_sizes_ok(int B, int Hkv, int page, int budget) {
  return B >= 1 && Hkv >= 1 && Hkv <= 4096 && B <= (1 << 20) &&
         (page == 16 || page == 32 || page == 64 || page == 128) &&
         budget >= 1 && budget <= (1 << 30) &&
         (long long)B * Hkv * 2 * ((budget + page - 1) / page) <= 0x7fffffffll;
}

// Workspace: the counter, the pages' flags, the kept slots.
size_t flags_at() { return 256; }
size_t kept_at(int B, int Hkv, int page, int budget) {
  const size_t pages = (budget + page - 1) / page;
  return flags_at() +
         ((size_t)B * Hkv * 2 * pages * sizeof(unsigned) + 255) / 256 * 256;
}

template <int kUnits>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
  PdlLaunch M(dim3((unsigned)((long long)a.pages * a.B * a.Hkv * 2)),
              dim3(kMove), 0, s);
  return cudaLaunchKernelEx(&M.cfg, kv_evict_move_kernel<kUnits>, a);
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_kv_evict_workspace_bytes(int B, int Hkv, int page, int budget) {
  using namespace dflash;
  if (!evict_sizes_ok(B, Hkv, page, budget)) return 0;
  const size_t need = kept_at(B, Hkv, page, budget) +
                      (size_t)B * Hkv * budget * sizeof(int);
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
  uint8_t* w = static_cast<uint8_t*>(ws);
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
  a.ticket = reinterpret_cast<unsigned*>(w);
  a.flags = reinterpret_cast<unsigned*>(w + flags_at());
  a.kept = kept ? kept
                : reinterpret_cast<int*>(w + kept_at(B, Hkv, page, budget));
  a.pages = (int)std::min<long long>((budget + page - 1) / page, max_pages);
  a.wait_ns = wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PdlLaunch S(dim3((unsigned)(B * Hkv)), dim3(kSelect), 0, s);
  cudaError_t e = cudaLaunchKernelEx(&S.cfg, kv_evict_select_kernel, a);
  if (e != cudaSuccess) return DFLASH_ERR_CUDA;
  const int units = (page * D / 16 + kMove - 1) / kMove;
  e = units <= 1   ? launch_move<1>(a, s)
      : units <= 2 ? launch_move<2>(a, s)
      : units <= 4 ? launch_move<4>(a, s)
      : units <= 8 ? launch_move<8>(a, s)
                   : launch_move<16>(a, s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
