// Attention of each sequence's last tokens over its paged 8-bit cache: the
// entry point, the CUDA-core kernel (fp32 storage, or heads wider than the
// tensor-core kernel takes) and the kernel that joins split sequences.
//
// Mathematics.  s_t = scale <q, k_t>; out = sum_t p_t v_t / l with
// p_t = exp(s_t - m), l = sum_t p_t, one pass over the tokens with the
// running maximum m (accumulators are multiplied by exp(m_old - m_new)).
// Two parts of a sequence with (m1, l1, o1), (m2, l2, o2) join as
// o = sum_i exp(m_i - m) o_i, l likewise, so a long sequence is cut into
// parts that run at the same time.
//
// A row is a (query, head) pair; the Hq / Hkv heads that share a key head
// read its tokens together.  The CUDA-core kernel takes 16 rows of one key
// head and a part of the tokens: tiles of 32 tokens go through registers
// (loaded one tile ahead) to shared memory as fp32; lane = token for the
// scores, lane = dimension for the sum of values.
#include <cuda_fp8.h>

#include <algorithm>

#include "kernels.h"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

constexpr int kRows = 16;     // rows of a CTA
constexpr int kTok = 32;      // tokens of a tile
constexpr int kWarps = 4;
constexpr int kRowsWarp = kRows / kWarps;
constexpr int kMaxSplits = 32;
constexpr int kTargetCtas = 608;  // four to an SM

// Parts each sequence is cut into, from the sizes the host knows.
int simt_splits(long long B, long long Q, int Hq, int Hkv) {
  const long long tiles = (Q * (Hq / Hkv) + kRows - 1) / kRows;
  const long long items = B * Hkv * tiles;
  const long long want = (kTargetCtas + items - 1) / items;
  return (int)std::min<long long>(want, kMaxSplits);
}

size_t simt_ws(long long B, long long Q, int Hq, int Hkv, int D) {
  const int ns = simt_splits(B, Q, Hq, Hkv);
  if (ns == 1) return 256;
  return (size_t)ns * B * Q * Hq * (D + 2) * sizeof(float);
}

// Values of the 16 codes of w times s, as fp32.
__device__ __forceinline__ void decode16(const uint4& w, float s,
                                         float (&f)[16]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(x[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 t = __half22float2(__half2(h));
    f[2 * i] = t.x * s;
    f[2 * i + 1] = t.y * s;
  }
}

// KD = 32-dimension slices of the widest head this instance takes.
template <typename T, int KD>
__global__ void __launch_bounds__(kWarps * 32)
    paged_attn_simt_kernel(const __grid_constant__ PagedAttnArgs a, int splits,
                           int row_tiles, float* __restrict__ part) {
  constexpr int DM = 32 * KD;
  constexpr int kChunks = kTok * DM / 16 / (kWarps * 32);  // per thread
  extern __shared__ float4 smem4[];
  float* sk = reinterpret_cast<float*>(smem4);      // [kTok][D + 4]
  const int D = a.D, SK = D + 4;
  float* sv = sk + kTok * SK;                       // [kTok][D]
  float* sq = sv + kTok * D;                        // [kRows][D]
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int item = blockIdx.x;
  const int sp = item % splits;
  item /= splits;
  const int tile = item % row_tiles;
  item /= row_tiles;
  const int hk = item % a.Hkv, b = item / a.Hkv;
  const int g = a.Hq / a.Hkv;
  bool bad = false;
  const int n = attn_clamp(a.kv_len[b], a.max_pages * (long long)a.page, &bad);
  const int nq = attn_clamp(a.q_len ? a.q_len[b] : a.Q, a.Q, &bad);
  if (bad && tid == 0) raise_error(a.err, kErrBadIndex);

  for (int i = tid; i < kRows * D; i += kWarps * 32) {
    const int r = tile * kRows + i / D;
    const int qi = r / g, h = hk * g + r % g;
    sq[i] = qi < nq ? to_f32(static_cast<const T*>(a.q)[
                          (((size_t)b * a.Q + qi) * a.Hq + h) * D + i % D]) *
                          a.scale
                    : 0.f;
  }
  // tokens each of this warp's rows sees: t < lim
  int lim[kRowsWarp];
  int most = 0;
#pragma unroll
  for (int k = 0; k < kRowsWarp; ++k) {
    const int r = tile * kRows + wid * kRowsWarp + k;
    const int qi = r / g;
    lim[k] = qi >= nq ? 0 : a.causal ? max(0, min(n, n - nq + qi + 1)) : n;
  }
  {
    const int r_last = min((tile + 1) * kRows, a.Q * g) - 1;
    const int qi = min(r_last / g, nq - 1);
    most = nq == 0 ? 0 : a.causal ? max(0, min(n, n - nq + qi + 1)) : n;
  }
  int chunk = (most + splits - 1) / splits;
  chunk = max((chunk + kTok - 1) / kTok * kTok, 2 * kTok);
  const int t0 = (int)min((long long)sp * chunk, (long long)most);
  const int t1 = (int)min((long long)t0 + chunk, (long long)most);

  uint4 kr[kChunks], vr[kChunks];
  float ks[kChunks], vs[kChunks];
  const int row_chunks = D / 16;
  auto fetch = [&](int base) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = tid + c * kWarps * 32;
      const int t = base + i / row_chunks;
      kr[c] = vr[c] = make_uint4(0, 0, 0, 0);
      ks[c] = vs[c] = 0.f;
      if (i < kTok * row_chunks && t < t1) {
        const int id = a.table[(size_t)b * a.max_pages + t / a.page];
        if (id >= 0 && id < a.num_pages) {
          const size_t ph = (size_t)id * a.Hkv + hk;
          const size_t at = (ph * a.page + t % a.page) * D +
                            (i % row_chunks) * 16;
          kr[c] = *reinterpret_cast<const uint4*>(a.k_codes + at);
          vr[c] = *reinterpret_cast<const uint4*>(a.v_codes + at);
          ks[c] = a.k_scale[ph];
          vs[c] = a.v_scale[ph];
        } else {
          raise_error(a.err, kErrBadIndex);
        }
      }
    }
  };
  float m[kRowsWarp], l[kRowsWarp], o[kRowsWarp][KD];
#pragma unroll
  for (int k = 0; k < kRowsWarp; ++k) {
    m[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int d = 0; d < KD; ++d) o[k][d] = 0.f;
  }
  if (t0 < t1) fetch(t0);
  for (int base = t0; base < t1; base += kTok) {
    __syncthreads();  // the previous tile has been read
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int i = tid + c * kWarps * 32;
      if (i < kTok * row_chunks) {
        const int t = i / row_chunks, d = (i % row_chunks) * 16;
        float f[16];
        decode16(kr[c], ks[c], f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(sk + t * SK + d + 4 * k) =
              make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
        decode16(vr[c], vs[c], f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<float4*>(sv + t * D + d + 4 * k) =
              make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
      }
    }
    __syncthreads();
    if (base + kTok < t1) fetch(base + kTok);
    float s[kRowsWarp] = {};
    const float* kt = sk + lane * SK;
    const float* qr = sq + wid * kRowsWarp * D;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      const float4 kv = *reinterpret_cast<const float4*>(kt + d);
#pragma unroll
      for (int k = 0; k < kRowsWarp; ++k) {
        const float4 qv = *reinterpret_cast<const float4*>(qr + k * D + d);
        s[k] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y,
                    fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[k]))));
      }
    }
    float p[kRowsWarp];
#pragma unroll
    for (int k = 0; k < kRowsWarp; ++k) {
      const bool sees = base + lane < min(lim[k], t1);
      const float x = sees ? s[k] : -INFINITY;
      const float mn = fmaxf(m[k], warp_max(x));
      const float f = mn == -INFINITY ? 1.f : expf(m[k] - mn);
      p[k] = x == -INFINITY ? 0.f : expf(x - mn);
      l[k] = l[k] * f + p[k];
      m[k] = mn;
#pragma unroll
      for (int d = 0; d < KD; ++d) o[k][d] *= f;
    }
#pragma unroll 4
    for (int t = 0; t < kTok; ++t) {
      float v[KD];
#pragma unroll
      for (int d = 0; d < KD; ++d)
        v[d] = lane + 32 * d < D ? sv[t * D + lane + 32 * d] : 0.f;
#pragma unroll
      for (int k = 0; k < kRowsWarp; ++k) {
        const float w = __shfl_sync(0xffffffffu, p[k], t);
#pragma unroll
        for (int d = 0; d < KD; ++d) o[k][d] = fmaf(w, v[d], o[k][d]);
      }
    }
  }
  const long long rows = (long long)a.B * a.Q * a.Hq;
#pragma unroll
  for (int k = 0; k < kRowsWarp; ++k) {
    const int r = tile * kRows + wid * kRowsWarp + k;
    const float sum = warp_sum(l[k]);
    if (r >= a.Q * g) continue;
    const long long row = ((long long)b * a.Q + r / g) * a.Hq + hk * g + r % g;
    if (splits == 1) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int d = 0; d < KD; ++d)
        if (lane + 32 * d < D)
          static_cast<T*>(a.out)[row * D + lane + 32 * d] =
              from_f32<T>(o[k][d] * inv);
      if (lane == 0 && a.lse)
        a.lse[row] = sum > 0.f ? m[k] + logf(sum) : -INFINITY;
    } else {
      float* po = part + ((size_t)sp * rows + row) * D;
      float* pm = part + (size_t)splits * rows * D + ((size_t)sp * rows + row) * 2;
#pragma unroll
      for (int d = 0; d < KD; ++d)
        if (lane + 32 * d < D) po[lane + 32 * d] = o[k][d];
      if (lane == 0) {
        pm[0] = m[k];
        pm[1] = sum;
      }
    }
  }
}

// One warp per row: the parts' (m, l, o) into out and lse.
template <typename T>
__global__ void __launch_bounds__(128)
    paged_attn_join_kernel(const float* __restrict__ part, int splits,
                           long long rows, int D, T* __restrict__ out,
                           float* __restrict__ lse) {
  pdl_trigger();
  pdl_wait();
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const float* pm = part + (size_t)splits * rows * D;
  float mi = -INFINITY, li = 0.f;
  if (lane < splits) {
    mi = pm[((size_t)lane * rows + row) * 2];
    li = pm[((size_t)lane * rows + row) * 2 + 1];
  }
  const float m = warp_max(mi);
  const float w = mi == -INFINITY ? 0.f : expf(mi - m);
  const float l = warp_sum(w * li);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int base = 0; base < D; base += 32) {  // whole warps shuffle
    const int d = base + lane;
    float o = 0.f;
    for (int s = 0; s < splits; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      if (d < D && ws != 0.f)
        o = fmaf(ws, part[((size_t)s * rows + row) * D + d], o);
    }
    if (d < D) out[row * D + d] = from_f32<T>(o * inv);
  }
  if (lane == 0 && lse) lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T, int KD>
cudaError_t launch_simt(const PagedAttnArgs& a, float* part, cudaStream_t s) {
  const int g = a.Hq / a.Hkv;
  const int tiles = (a.Q * g + kRows - 1) / kRows;
  const int ns = simt_splits(a.B, a.Q, a.Hq, a.Hkv);
  const long long ctas = (long long)a.B * a.Hkv * tiles * ns;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  const size_t smem = (size_t)(kTok * (a.D + 4) + kTok * a.D + kRows * a.D) *
                      sizeof(float);
  auto* f = paged_attn_simt_kernel<T, KD>;
  cudaError_t e = cudaFuncSetAttribute(
      f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3((unsigned)ctas), dim3(kWarps * 32), smem, s);
  e = cudaLaunchKernelEx(&L.cfg, f, a, ns, tiles, part);
  if (e != cudaSuccess || ns == 1) return e;
  const long long rows = (long long)a.B * a.Q * a.Hq;
  PdlLaunch J(dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s);
  return cudaLaunchKernelEx(&J.cfg, paged_attn_join_kernel<T>,
                            (const float*)part, ns, rows, a.D,
                            static_cast<T*>(a.out), a.lse);
}

template <typename T>
cudaError_t launch_simt_d(const PagedAttnArgs& a, float* part,
                          cudaStream_t s) {
  if (a.D <= 64) return launch_simt<T, 2>(a, part, s);
  if (a.D <= 128) return launch_simt<T, 4>(a, part, s);
  return launch_simt<T, 8>(a, part, s);
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool attn_sizes_ok(int B, int Q, int Hq, int Hkv, int D) {
  return cache_sizes_ok(B, Q, Hq, Hkv, D, 16, 1, 1) && Hq / Hkv <= 64;
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_paged_attn_workspace_bytes(int B, int Q, int Hq, int Hkv,
                                         int D) {
  using namespace dflash;
  if (!attn_sizes_ok(B, Q, Hq, Hkv, D)) return 0;
  // an upper bound over both dtypes
  size_t need = simt_ws(B, Q, Hq, Hkv, D);
  if (paged_attn_tc_takes(D, DFLASH_BF16))
    need = std::max(need, paged_attn_tc_ws(B, Q, Hq, Hkv));
  return (need + 255) & ~(size_t)255;
}

dflash_status dflash_paged_attn(
    const void* q, const uint8_t* k_codes, const uint8_t* v_codes,
    const float* k_scale, const float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, const int32_t* q_len, int B, int Q, int Hq,
    int Hkv, int D, int page, int num_pages, int max_pages, int causal,
    float scale, dflash_dtype dt, void* out, float* lse, void* ws,
    size_t ws_bytes, dflash_stream_t stream) {
  using namespace dflash;
  if (!(q && k_codes && v_codes && k_scale && v_scale && page_table &&
        kv_len && out && ws))
    return DFLASH_ERR_INVALID_ARG;
  if (dt != DFLASH_BF16 && dt != DFLASH_FP32) return DFLASH_ERR_INVALID_ARG;
  if (!cache_sizes_ok(B, Q, Hq, Hkv, D, page, num_pages, max_pages) ||
      !attn_sizes_ok(B, Q, Hq, Hkv, D))
    return DFLASH_ERR_INVALID_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(k_codes, 16) ||
      !aligned_to(v_codes, 16) || !aligned_to(ws, 256))
    return DFLASH_ERR_INVALID_ARG;
  if (ws_bytes < dflash_paged_attn_workspace_bytes(B, Q, Hq, Hkv, D))
    return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  PagedAttnArgs a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.q = q;
  a.k_codes = k_codes;
  a.v_codes = v_codes;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = page_table;
  a.kv_len = kv_len;
  a.q_len = q_len;
  a.B = B;
  a.Q = Q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.causal = causal != 0;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      paged_attn_tc_takes(D, dt)
          ? launch_paged_attn_tc(a, sms, static_cast<float*>(ws), s)
      : dt == DFLASH_FP32
          ? launch_simt_d<float>(a, static_cast<float*>(ws), s)
          : launch_simt_d<__nv_bfloat16>(a, static_cast<float*>(ws), s);
  return e == cudaSuccess ? DFLASH_OK : DFLASH_ERR_CUDA;
}

}  // extern "C"
