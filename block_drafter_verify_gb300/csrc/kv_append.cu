// Appending a block's keys and values to the paged 8-bit cache, with the
// position rotation of q and k on the way.
//
// Mathematics.  A pair (a, b) of a head turns by the angle of its position,
// (a c - b s, b c + a s).  A page of tokens and one key head share one scale,
// a power of two: E4M3 is a floating-point format, so such a scale costs no
// precision of the codes, and when a page's scale has to grow because a
// louder token arrives, the older codes move to it exactly (their exponent
// drops), except those that become subnormal.  Products and sums of the
// rotation are rounded separately (no contraction), so the codes are a
// function of the inputs alone.
//
// One launch, two kinds of CTA.  Cache CTAs own one (sequence, touched page,
// key head, k or v): they see every new token of the page, so the maximum,
// the scale, the older codes' rewrite and the new codes need no second
// launch and no atomics.  Rotation CTAs take tokens of q; a thread keeps its
// angles for up to kHeads heads.
//
// Bound: bytes (each value is read once and held in registers between the
// maximum and the conversion); at decode sizes the launch itself (3 to 7 us on
// the GPU).  Four prompts of 13000 tokens in all, 32 + 8 heads of 128, bf16:
// 59 us for 324 MB, 5.5 TB/s.  The cache's CTAs alone take 27 us (12 us of
// bytes: they wait for lengths, page ids, values and each other), which the
// rotation's traffic fills where both alternate; one kind after the other took
// 69 us.  Three CTAs to an SM: two 80 us, four (64 registers) 72 us.
#include <cuda_fp8.h>

#include "kernels.h"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

constexpr int kMinExp = -64;   // smallest exponent of a block scale
constexpr int kThreads = 256;  // most threads of a CTA
constexpr int kKeep = 2;       // units a thread keeps in registers
constexpr int kHeads = 8;      // q heads per rotation thread

// Division of numbers below 2^31 by d: with 2^(s-1) < d <= 2^s and
// m = ceil(2^(31+s) / d), n m / 2^(31+s) exceeds n / d by less than
// n / 2^31 / d, so its integer part is n / d's.  A division by a variable
// takes some 25 instructions, and a thread that appends has only 32 values.
struct Div {
  uint32_t d, m, s;
  Div() = default;
  explicit Div(uint32_t by) : d(by), m(0), s(0) {
    while ((1ull << s) < by) ++s;
    if (s > 0) m = (uint32_t)(((1ull << (31 + s)) + by - 1) / by);
  }
  __device__ __forceinline__ int of(int n) const {
    return s > 0 ? (int)(__umulhi((uint32_t)n, m) >> (s - 1)) : n;
  }
  // n / d, and n to what remains
  __device__ __forceinline__ int split(int& n) const {
    const int q = of(n);
    n -= q * (int)d;
    return q;
  }
};

struct AppendArgs {
  const void* x[2];           // k, v
  long long ld[2];
  const void* q;
  long long ld_q;
  const float *cos_tab, *sin_tab;
  const int *pos, *n_new, *table;
  int B, Q, Hq, Hkv, D, rot, max_pos, page, num_pages, max_pages;
  void* q_out;
  uint8_t* codes[2];
  float* scale[2];
  int* kv_len;
  int touched;                // most pages a sequence's tokens fall into
  uint32_t share;  // of the grid, the CTAs of the cache
  int rotates;     // there are others
  Div groups, units, heads, seqs, block, pages;  // kHeads' of Hq, ..., page
  int* err;
};

// N values of type T (4 or 8) as loaded.
template <typename T, int N>
struct Raw {
  static_assert(N == 4 || N == 8, "");
  static constexpr int W = N * sizeof(T) / 4;  // 32-bit words
  uint32_t w[W];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&f)[N]) {
  Raw<T, N> r;
  r.load(p);
  r.get(f);
}

template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&f)[N]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) =
          make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// A unit is the 2 VEC values of one head that one thread turns: with
// half-split pairs dimensions [j, j + VEC) and [j + rot/2, ...), otherwise
// (interleaved, or past the rotated dimensions) 2 VEC consecutive ones.
struct Unit {
  int d0, d1;   // first dimension of each half
  int angle;    // first angle, -1 past the rotated dimensions
};
template <int VEC, bool kInter>
__device__ __forceinline__ Unit unit_at(int u, int rot) {
  if (2 * VEC * u < rot) {
    if constexpr (kInter) return Unit{2 * VEC * u, 2 * VEC * u + VEC, VEC * u};
    return Unit{VEC * u, VEC * u + rot / 2, VEC * u};
  }
  return Unit{2 * VEC * u, 2 * VEC * u + VEC, -1};
}

template <int VEC, bool kInter>
__device__ __forceinline__ void rotate(float (&a)[VEC], float (&b)[VEC],
                                       const float (&c)[VEC],
                                       const float (&s)[VEC]) {
  if constexpr (kInter) {
    // angle i turns consecutive values 2i, 2i + 1 of the unit (a, then b)
    float x[2 * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) { x[i] = a[i]; x[VEC + i] = b[i]; }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float p = x[2 * i], r = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(r, s[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(r, c[i]), __fmul_rn(p, s[i]));
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) { a[i] = x[i]; b[i] = x[VEC + i]; }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float p = a[i], r = b[i];
      a[i] = __fsub_rn(__fmul_rn(p, c[i]), __fmul_rn(r, s[i]));
      b[i] = __fadd_rn(__fmul_rn(r, c[i]), __fmul_rn(p, s[i]));
    }
  }
}

// Exponent of the least power of two s with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t w = __float_as_uint(amax);
  if (w < 0x00800000u) return kMinExp;  // zero or subnormal
  const int e = (int)(w >> 23) - 127 - 8 + ((w & 0x7fffffu) > 0x600000u);
  return e < kMinExp ? kMinExp : e;
}
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

template <int VEC>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&f)[VEC],
                                            float inv) {
  uint32_t w[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = f[4 * i + k] * inv;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[0], t[1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[2], t[3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  if constexpr (VEC == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(p) = w[0];
}

// Two codes times a power of two, rounded to codes again.
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

// New tokens of sequence b that fit: clamped to the tables; *bad if not all.
__device__ __forceinline__ int live_tokens(const AppendArgs& a, int b,
                                           int* pos_out, bool* bad) {
  const int pos = a.pos[b];
  const int n = a.n_new ? a.n_new[b] : a.Q;
  *pos_out = pos;
  *bad = false;
  if (pos < 0 || n < 0 || n > a.Q) {
    *bad = true;
    return 0;
  }
  long long most = (long long)a.max_pages * a.page;
  if (a.rot > 0 && a.max_pos < most) most = a.max_pos;
  const long long room = most - pos;
  if (n > room) {
    *bad = true;
    return room > 0 ? (int)room : 0;
  }
  return n;
}

template <typename T, int VEC, bool kInter>
__global__ void __launch_bounds__(kThreads, 3)
    kv_append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, nt = blockDim.x;
  const int units = a.D / (2 * VEC);
  const int r2 = a.rot / 2;
  // The CTAs of both kinds alternate evenly, so that the rotation's traffic
  // fills the waits of the cache's: of the first x, x share / 2^32 are the
  // cache's (share: the part of 2^32, rounded up, that they are of the grid).
  const uint32_t x = blockIdx.x, before = __umulhi(x, a.share);
  if (a.rotates && __umulhi(x + 1, a.share) == before) {
    // ---- rotation of q ---------------------------------------------------
    int hg = (int)(x - before);
    const int i = a.groups.split(hg) * nt + tid;
    if (i >= a.B * a.Q * units) return;
    int u = i;
    const int row_of = a.units.split(u);
    int j = row_of;
    const int b = a.block.split(j);
    const long long row = row_of;
    int pos;
    bool bad;
    const bool live = j < live_tokens(a, b, &pos, &bad);
    const Unit un = unit_at<VEC, kInter>(u, a.rot);
    float c[VEC], s[VEC];
    if (live && un.angle >= 0) {
      const size_t at = (size_t)(pos + j) * r2 + un.angle;
      load_n<float, VEC>(a.cos_tab + at, c);
      load_n<float, VEC>(a.sin_tab + at, s);
    }
    const T* src = static_cast<const T*>(a.q) + row * a.ld_q;
    T* dst = static_cast<T*>(a.q_out) + row * a.Hq * a.D;
    const int h1 = min(a.Hq, (hg + 1) * kHeads);
    for (int h0 = hg * kHeads; h0 < h1; h0 += 4) {  // four heads in flight
      Raw<T, VEC> x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (live && h0 + i < h1) {
          x[i].load(src + (size_t)(h0 + i) * a.D + un.d0);
          y[i].load(src + (size_t)(h0 + i) * a.D + un.d1);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (h0 + i >= h1) break;
        float u[VEC] = {}, v[VEC] = {};
        if (live) {
          x[i].get(u);
          y[i].get(v);
          if (un.angle >= 0) rotate<VEC, kInter>(u, v, c, s);
        }
        store_n<T, VEC>(dst + (size_t)(h0 + i) * a.D + un.d0, u);
        store_n<T, VEC>(dst + (size_t)(h0 + i) * a.D + un.d1, v);
      }
    }
    return;
  }
  // ---- one page and head of k or v ---------------------------------------
  int h = a.rotates ? (int)before : (int)x;
  const int kv = h & 1;
  h >>= 1;
  int b = a.heads.split(h);
  const int t = a.seqs.split(b);
  int pos;
  bool bad;
  const int n = live_tokens(a, b, &pos, &bad);
  if (t == 0 && h == 0 && kv == 0 && tid == 0) {
    a.kv_len[b] = pos + n;
    if (bad) raise_error(a.err, kErrBadIndex);
  }
  if (n == 0) return;
  const int pg = a.pages.of(pos) + t;          // page of the sequence
  const long long start = (long long)pg * a.page;
  const long long end = (long long)pos + n;
  if (start >= end) return;
  const int id = a.table[(size_t)b * a.max_pages + pg];
  const int first = pos > start ? (int)(pos - start) : 0;  // older tokens
  const int last = (int)(end - start < a.page ? end - start : a.page);
  const int work = (last - first) * units;
  const bool turn = kv == 0 && a.rot > 0;
  const T* src = static_cast<const T*>(a.x[kv]) +
                 ((long long)b * a.Q + (start + first - pos)) * a.ld[kv] +
                 (size_t)h * a.D;
  uint8_t* dst = nullptr;
  auto fetch = [&](int i, float (&x)[VEC], float (&y)[VEC]) {
    int u = i;
    const int j = a.units.split(u);
    const Unit un = unit_at<VEC, kInter>(u, a.rot);
    const T* p = src + (long long)j * a.ld[kv];
    load_n<T, VEC>(p + un.d0, x);
    load_n<T, VEC>(p + un.d1, y);
    if (turn && un.angle >= 0) {
      float c[VEC], s[VEC];
      const size_t at = (size_t)(start + first + j) * r2 + un.angle;
      load_n<float, VEC>(a.cos_tab + at, c);
      load_n<float, VEC>(a.sin_tab + at, s);
      rotate<VEC, kInter>(x, y, c, s);
    }
  };
  bool odd = false;  // a value of this thread's is not finite
  auto put = [&](int i, const float (&x)[VEC], const float (&y)[VEC],
                 float inv) {
    int u = i;
    const int j = a.units.split(u);
    const Unit un = unit_at<VEC, kInter>(u, a.rot);
    uint8_t* p = dst + (size_t)(first + j) * a.D;
    store_codes<VEC>(p + un.d0, x, inv);
    store_codes<VEC>(p + un.d1, y, inv);
  };
  float top = 0.f;  // a NaN stays one
  auto fold = [&](const float (&x)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(x[k])));
  };
  float amax = 0.f;
  auto fold_finite = [&](const float (&x)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (fabsf(x[k]) < INFINITY) amax = fmaxf(amax, fabsf(x[k]));
  };
  auto no_nan = [](float (&x)[VEC]) {  // a NaN is stored as 0
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (x[k] != x[k]) x[k] = 0.f;
  };
  float xs[kKeep][VEC], ys[kKeep][VEC];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = tid + k * nt;
    if (i < work) {
      fetch(i, xs[k], ys[k]);
      fold(xs[k]);
      fold(ys[k]);
    }
  }
  for (int i = tid + kKeep * nt; i < work; i += nt) {  // larger pages
    float p[VEC], r[VEC];
    fetch(i, p, r);
    fold(p);
    fold(r);
  }
  if (top < INFINITY) {
    amax = top;
  } else {
    odd = true;
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (tid + k * nt < work) {
        fold_finite(xs[k]);
        fold_finite(ys[k]);
        no_nan(xs[k]);
        no_nan(ys[k]);
      }
    for (int i = tid + kKeep * nt; i < work; i += nt) {
      float p[VEC], r[VEC];
      fetch(i, p, r);
      fold_finite(p);
      fold_finite(r);
    }
  }
  __shared__ float s_max[kThreads / 32];
  amax = warp_max(amax);
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  // only now: the values travelled meanwhile
  if (id < 0 || id >= a.num_pages) {  // uniform
    if (tid == 0) raise_error(a.err, kErrBadIndex);
    return;
  }
  dst = a.codes[kv] + ((size_t)id * a.Hkv + h) * a.page * a.D;
  float* scale = a.scale[kv] + (size_t)id * a.Hkv + h;
  if (odd) raise_error(a.err, kErrNonfinite);
  const float was = first > 0 ? *scale : 0.f;
  __syncthreads();  // every thread has read the old scale, too
  for (int w = 0; w < (nt >> 5); ++w) amax = fmaxf(amax, s_max[w]);
  const float fresh = pow2(scale_exponent(amax));
  const float now = first > 0 ? fmaxf(was, fresh) : fresh;
  if (tid == 0) *scale = now;
  // now is a power of two unless the caller's own old scale is not
  const float inv = __frcp_rn(now);
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = tid + k * nt;
    if (i < work) put(i, xs[k], ys[k], inv);
  }
  for (int i = tid + kKeep * nt; i < work; i += nt) {
    float p[VEC], r[VEC];
    fetch(i, p, r);
    if (odd) {
      no_nan(p);
      no_nan(r);
    }
    put(i, p, r, inv);
  }
  if (first > 0 && now != was) {
    const float ratio = __fdiv_rn(was, now);
    uint4* old = reinterpret_cast<uint4*>(dst);  // D % 16 == 0
    for (int i = tid; i < first * a.D / 16; i += nt) {
      uint4 w = old[i];
      w.x = requant4(w.x, ratio);
      w.y = requant4(w.y, ratio);
      w.z = requant4(w.z, ratio);
      w.w = requant4(w.w, ratio);
      old[i] = w;
    }
  }
}

template <typename T, int VEC>
cudaError_t launch(const AppendArgs& a, bool inter, cudaStream_t s) {
  AppendArgs args = a;
  const int units = a.D / (2 * VEC);
  const long long most = (long long)(a.Q < a.page ? a.Q : a.page) * units;
  int nt = (int)(most < kThreads ? (most + 31) / 32 * 32 : kThreads);
  if (nt < 64) nt = 64;
  const long long cache = 2ll * a.Hkv * a.B * a.touched;
  long long rot = 0;
  if (a.q)
    rot = (((long long)a.B * a.Q * units + nt - 1) / nt) *
          ((a.Hq + kHeads - 1) / kHeads);
  if (cache + rot > 0x7fffffffll ||
      (a.q && (long long)a.B * a.Q * units > 0x7fffffffll - kThreads))
    return cudaErrorNotSupported;
  // (cache + rot is below 2^31: the rounding up adds less than a half)
  args.rotates = rot > 0;
  args.groups = Div(a.q ? (a.Hq + kHeads - 1) / kHeads : 1);
  args.units = Div(units);
  args.heads = Div(a.Hkv);
  args.seqs = Div(a.B);
  args.block = Div(a.Q);
  args.pages = Div(a.page);
  args.share = (uint32_t)((((unsigned long long)cache << 32) + cache + rot - 1) /
                          (unsigned long long)(cache + rot));
  PdlLaunch L(dim3((unsigned)(cache + rot)), dim3(nt), 0, s);
  return inter ? cudaLaunchKernelEx(&L.cfg, kv_append_kernel<T, VEC, true>, args)
               : cudaLaunchKernelEx(&L.cfg, kv_append_kernel<T, VEC, false>, args);
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace
}  // namespace dflash

extern "C" dflash_status dflash_kv_append(
    const void* q, const void* k, const void* v, int64_t ld_q, int64_t ld_k,
    int64_t ld_v, const float* cos_tab, const float* sin_tab,
    const int32_t* pos, const int32_t* n_new, const int32_t* page_table,
    int B, int Q, int Hq, int Hkv, int D, int rot, int interleaved,
    int max_pos, int page, int num_pages, int max_pages, dflash_dtype dt,
    void* q_out, uint8_t* k_codes, uint8_t* v_codes, float* k_scale,
    float* v_scale, int32_t* kv_len, dflash_stream_t stream) {
  using namespace dflash;
  if (!(k && v && pos && page_table && k_codes && v_codes && k_scale &&
        v_scale && kv_len) || kv_len == pos)
    return DFLASH_ERR_INVALID_ARG;
  if (q && !q_out) return DFLASH_ERR_INVALID_ARG;
  if (dt != DFLASH_BF16 && dt != DFLASH_FP32) return DFLASH_ERR_INVALID_ARG;
  if (!cache_sizes_ok(B, Q, q ? Hq : Hkv, Hkv, D, page, num_pages, max_pages))
    return DFLASH_ERR_INVALID_ARG;
  if (rot < 0 || rot > D || rot % 8 != 0) return DFLASH_ERR_INVALID_ARG;
  if (rot > 0 && (!cos_tab || !sin_tab || max_pos < 1))
    return DFLASH_ERR_INVALID_ARG;
  const uintptr_t four = dt == DFLASH_FP32 ? 16 : 8;  // bytes of 4 elements
  if (ld_k < (int64_t)Hkv * D || ld_v < (int64_t)Hkv * D || ld_k % 4 ||
      ld_v % 4 || !aligned_to(k, four) || !aligned_to(v, four))
    return DFLASH_ERR_INVALID_ARG;
  if (q && (ld_q < (int64_t)Hq * D || ld_q % 4 || !aligned_to(q, four) ||
            !aligned_to(q_out, four)))
    return DFLASH_ERR_INVALID_ARG;
  if (!aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) ||
      (rot > 0 && (!aligned_to(cos_tab, 16) || !aligned_to(sin_tab, 16))))
    return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  AppendArgs a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.x[0] = k;
  a.x[1] = v;
  a.ld[0] = ld_k;
  a.ld[1] = ld_v;
  a.q = q;
  a.ld_q = ld_q;
  a.cos_tab = cos_tab;
  a.sin_tab = sin_tab;
  a.pos = pos;
  a.n_new = n_new;
  a.table = page_table;
  a.B = B;
  a.Q = Q;
  a.Hq = q ? Hq : 0;
  a.Hkv = Hkv;
  a.D = D;
  a.rot = rot;
  a.max_pos = max_pos;
  a.page = page;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.q_out = q_out;
  a.codes[0] = k_codes;
  a.codes[1] = v_codes;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.kv_len = kv_len;
  a.touched = (Q - 1) / page + 2;
  if (a.touched > max_pages) a.touched = max_pages;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  // Eight values to a load where rot, the rows and the pointers allow it
  // (16 bytes of bf16), four otherwise.
  const bool wide =
      dt == DFLASH_BF16 && rot % 16 == 0 && ld_k % 8 == 0 && ld_v % 8 == 0 &&
      aligned_to(k, 16) && aligned_to(v, 16) &&
      (!q || (ld_q % 8 == 0 && aligned_to(q, 16) && aligned_to(q_out, 16)));
  if (dt == DFLASH_FP32)
    e = launch<float, 4>(a, interleaved != 0, s);
  else if (wide)
    e = launch<__nv_bfloat16, 8>(a, interleaved != 0, s);
  else
    e = launch<__nv_bfloat16, 4>(a, interleaved != 0, s);
  return e == cudaSuccess            ? DFLASH_OK
         : e == cudaErrorNotSupported ? DFLASH_ERR_UNSUPPORTED
                                      : DFLASH_ERR_CUDA;
}
