// The attention weight that cached tokens gather: the entry point and the
// CUDA-core kernel (fp32 storage, or heads wider than the tensor-core kernel
// takes).
//
// Mathematics.  A token's weight for a row (a query and a head) is
// exp(s - lse), s = scale <q, k>, where lse is the row's logsumexp that the
// attention left: no second pass over the row, and tokens are independent.  So
// one CTA owns a tile of tokens of one sequence and key head and takes all of
// its rows in turn; the sum needs no atomics, and its order is fixed.
#include <cuda_fp8.h>

#include "kernels.h"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

constexpr int kTokens = 128;   // of a CTA, one a thread
constexpr int kRows = 8;       // rows at a time

template <typename T>
__global__ void __launch_bounds__(kTokens)
    attn_mass_simt_kernel(const __grid_constant__ AttnMassArgs a, int tiles) {
  __shared__ float4 s_q4[kRows * 256 / 4];
  __shared__ float s_lse[kRows];
  __shared__ int s_lim[kRows];
  float* s_q = reinterpret_cast<float*>(s_q4);
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, D = a.D;
  int item = blockIdx.x;
  const int tile = item % tiles;
  item /= tiles;
  const int hk = item % a.Hkv, b = item / a.Hkv;
  const int g = a.Hq / a.Hkv;
  bool bad = false;
  const int n = mass_length(a, b, &bad);
  const int nq = attn_clamp(a.q_len ? a.q_len[b] : a.Q, a.Q, &bad);
  if (bad && tid == 0) raise_error(a.err, kErrBadIndex);
  const int first = a.first / kTokens * kTokens;  // of the first tile
  const int base = first + tile * kTokens, t = base + tid;
  if (base >= n) return;
  const bool mine = t >= a.first && t < n;
  const uint8_t* key = nullptr;
  float ks = 0.f;
  if (mine) {
    const int id = a.table[(size_t)b * a.max_pages + t / a.page];
    if (id < 0 || id >= a.num_pages) {
      raise_error(a.err, kErrBadIndex);
    } else {
      const size_t ph = (size_t)id * a.Hkv + hk;
      key = a.k_codes + (ph * a.page + t % a.page) * D;
      ks = a.k_scale[ph];
    }
  }
  float sum = 0.f;
  const int rows = nq * g;
  // the first row that sees a token of the tile
  const int r0 = a.causal ? max(0, base - (n - nq)) * g / kRows * kRows : 0;
  for (int row0 = r0; row0 < rows; row0 += kRows) {
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kTokens) {
      const int r = row0 + i / D;
      s_q[i] = r < rows
                   ? to_f32(static_cast<const T*>(
                         a.q)[(((size_t)b * a.Q + r / g) * a.Hq + hk * g +
                               r % g) * D + i % D]) * a.scale
                   : 0.f;
    }
    if (tid < kRows) {
      const int r = row0 + tid;
      s_lse[tid] = r < rows ? a.lse[((size_t)b * a.Q + r / g) * a.Hq +
                                    hk * g + r % g]
                            : -INFINITY;
      s_lim[tid] = a.causal ? n - nq + r / g + 1 : n;
    }
    __syncthreads();
    if (!mine) continue;
    float s[kRows] = {};
    for (int d = 0; d < D; d += 16) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (key) w = *reinterpret_cast<const uint4*>(key + d);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
      float k[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(x[i >> 1] >> (16 * (i & 1))), __NV_E4M3)));
        k[2 * i] = f.x;
        k[2 * i + 1] = f.y;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float4* q = reinterpret_cast<const float4*>(s_q + r * D + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[r] = fmaf(q[i].x, k[4 * i], fmaf(q[i].y, k[4 * i + 1],
                 fmaf(q[i].z, k[4 * i + 2], fmaf(q[i].w, k[4 * i + 3],
                                                 s[r]))));
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (t < s_lim[r] && fabsf(s_lse[r]) != INFINITY)
        sum += expf(s[r] * ks - s_lse[r]);
  }
  if (mine) mass_store(a, b, hk, t, sum);
}

template <typename T>
cudaError_t launch_simt(const AttnMassArgs& a, cudaStream_t s) {
  const long long most = mass_most(a);
  const long long tiles =
      (most - a.first / kTokens * kTokens + kTokens - 1) / kTokens;
  const long long ctas = tiles * a.Hkv * a.B;
  if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
  PdlLaunch L(dim3((unsigned)ctas), dim3(kTokens), 0, s);
  return cudaLaunchKernelEx(&L.cfg, attn_mass_simt_kernel<T>, a, (int)tiles);
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace
}  // namespace dflash

extern "C" dflash_status dflash_attn_mass(
    const void* q, const uint8_t* k_codes, const float* k_scale,
    const int32_t* page_table, const int32_t* kv_len, const int32_t* q_len,
    const float* lse, const int32_t* fresh, int first, int B, int Q, int Hq,
    int Hkv, int D, int page, int num_pages, int max_pages, int causal,
    float scale, float decay, dflash_dtype dt, float* mass, int64_t ld_mass,
    dflash_stream_t stream) {
  using namespace dflash;
  if (!(q && k_codes && k_scale && page_table && kv_len && lse && mass))
    return DFLASH_ERR_INVALID_ARG;
  if (dt != DFLASH_BF16 && dt != DFLASH_FP32) return DFLASH_ERR_INVALID_ARG;
  if (!cache_sizes_ok(B, Q, Hq, Hkv, D, page, num_pages, max_pages) ||
      Hq / Hkv > 64 || (long long)B * Q * Hq > 0x7fffffffll)
    return DFLASH_ERR_INVALID_ARG;
  if (first < 0 || ld_mass < 1 || !(scale > -INFINITY && scale < INFINITY) ||
      !(decay > -INFINITY && decay < INFINITY))
    return DFLASH_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_codes, 16))
    return DFLASH_ERR_INVALID_ARG;
  int sms = 0;
  AttnMassArgs a;
  const dflash_status st = current_device_info(&sms, &a.err);
  if (st != DFLASH_OK) return st;
  a.q = q;
  a.k_codes = k_codes;
  a.k_scale = k_scale;
  a.table = page_table;
  a.kv_len = kv_len;
  a.q_len = q_len;
  a.lse = lse;
  a.fresh = fresh;
  a.first = first;
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
  a.decay = decay;
  a.mass = mass;
  a.ld_mass = ld_mass;
  a.wait_ns = wait_limit_ns();
  if (a.first >= mass_most(a)) return DFLASH_OK;  // no token to take
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = paged_attn_tc_takes(D, dt)
                            ? launch_attn_mass_tc(a, sms, s)
                        : dt == DFLASH_FP32 ? launch_simt<float>(a, s)
                                            : launch_simt<__nv_bfloat16>(a, s);
  return e == cudaSuccess            ? DFLASH_OK
         : e == cudaErrorNotSupported ? DFLASH_ERR_UNSUPPORTED
                                      : DFLASH_ERR_CUDA;
}
