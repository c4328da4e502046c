// Attention of a batch whose sequences share their first tokens: the entry
// point, and the launches of the CUDA-core kernel.
//
// Mathematics.  A row's softmax over the shared tokens and over its sequence's
// own are two parts of one softmax, (m, l, o) each, which join as the parts of a
// cut sequence do.  So the shared tokens are read with the rows of all sequences
// together: once from memory, and as many rows to a tile as there are.
#include <algorithm>

#include "attn_simt.cuh"
#include "kernels.h"

namespace dflash {

// SM count and device error word of the current device (api.cu).
dflash_status current_device_info(int* sms, int** err);

namespace {

// Two to an SM of 152.  Not the device's count: the workspace query has none.
constexpr int kTargetCtas = 304;
// Of the own tokens, where there are shared ones, too: those of a wave that the
// longer parts of the shared tokens leave, at least.
constexpr int kOwnCtas = 100;
constexpr int kMostSplits = kMaxSplits / 2;  // of the shared tokens, of others

struct Splits {
  long long own_tiles, shared_tiles;
  int own, shared;
};
// Parts that tokens are cut into.  The shared tokens' CTAs do not pass a wave.
// (fp32, 32 query and 8 key heads of 128: 16 sequences, 4096 shared tokens, four
// parts in 256 CTAs 101 us, five in 320 163, three 142; 5 sequences of 4 queries,
// 12 heads of 64, 1040 shared tokens 29 us, with 304 CTAs for either 37.  The rule
// does not see how many tokens are whose: one sequence, 16 shared tokens and 60000
// own ones 360 us, none shared 295.)
Splits simt_splits(long long B, long long Q, int Hq, int Hkv, bool any) {
  Splits s;
  s.own_tiles = (Q * (Hq / Hkv) + kRows - 1) / kRows;
  s.shared_tiles = (B * Q * (Hq / Hkv) + kRows - 1) / kRows;
  const long long items = B * Hkv * s.own_tiles;
  const int most = any ? kOwnCtas : kTargetCtas;
  s.own = (int)std::min<long long>((most + items - 1) / items, kMostSplits);
  s.shared = !any ? 0
                  : (int)std::min<long long>(
                        std::max(1ll, kTargetCtas / (Hkv * s.shared_tiles)),
                        kMostSplits);
  return s;
}

size_t simt_ws(long long B, long long Q, int Hq, int Hkv, int D) {
  int parts = 0;
  for (const bool any : {false, true}) {
    const Splits s = simt_splits(B, Q, Hq, Hkv, any);
    parts = std::max(parts, s.own + s.shared);
  }
  return (size_t)parts * B * Q * Hq * (D + 2) * sizeof(float);
}

template <typename T, int W, int G>
cudaError_t launch_simt(const PagedAttnArgs& a, int shared, float* part,
                        cudaStream_t s) {
  const Splits n = simt_splits(a.B, a.Q, a.Hq, a.Hkv, shared > 0);
  SharedView v{shared, n.shared, (int)n.shared_tiles, 0};
  if (shared > 0) {
    const long long items = a.Hkv * n.shared_tiles * n.shared;
    if (items > 0x7fffffffll) return cudaErrorNotSupported;
    v.items = (unsigned)items;
  }
  const long long ctas = v.items + a.B * a.Hkv * n.own_tiles * n.own;
  if (ctas > 0x7fffffffll) return cudaErrorNotSupported;
  const size_t smem = (size_t)(1 + kWarps) * kRows * a.D * sizeof(float);
  auto* f = paged_attn_simt_kernel<T, W, G, 2, true>;
  cudaError_t e = cudaFuncSetAttribute(
      f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  PdlLaunch L(dim3((unsigned)ctas), dim3(kWarps * 32), smem, s);
  e = cudaLaunchKernelEx(&L.cfg, f, a, n.own, (int)n.own_tiles, part, v);
  const int parts = v.splits + n.own;
  if (e != cudaSuccess || parts == 1) return e;
  const long long rows = (long long)a.B * a.Q * a.Hq;
  PdlLaunch J(dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s);
  return cudaLaunchKernelEx(&J.cfg, paged_attn_join_kernel<T>,
                            (const float*)part, parts, rows, a.D,
                            static_cast<T*>(a.out), a.lse);
}

template <typename T>
cudaError_t launch_simt_d(const PagedAttnArgs& a, int shared, float* part,
                          cudaStream_t s) {
  if (a.D <= 64) return launch_simt<T, 1, 2>(a, shared, part, s);
  if (a.D <= 128) return launch_simt<T, 1, 1>(a, shared, part, s);
  return launch_simt<T, 2, 1>(a, shared, part, s);
}

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

bool shared_sizes_ok(int B, int Q, int Hq, int Hkv, int D) {
  return cache_sizes_ok(B, Q, Hq, Hkv, D, 16, 1, 1) && Hq / Hkv <= 64 &&
         (long long)B * Q * Hq <= 0x7fffffffll;
}

}  // namespace
}  // namespace dflash

extern "C" {

size_t dflash_shared_attn_workspace_bytes(int B, int Q, int Hq, int Hkv,
                                          int D) {
  using namespace dflash;
  if (!shared_sizes_ok(B, Q, Hq, Hkv, D)) return 0;
  // an upper bound over both dtypes
  size_t need = simt_ws(B, Q, Hq, Hkv, D);
  if (paged_attn_tc_takes(D, DFLASH_BF16))
    need = std::max(need, shared_attn_tc_ws(B, Q, Hq, Hkv, D));
  return (need + 255) & ~(size_t)255;
}

dflash_status dflash_shared_attn(
    const void* q, const uint8_t* k_codes, const uint8_t* v_codes,
    const float* k_scale, const float* v_scale, const int32_t* page_table,
    const int32_t* kv_len, const int32_t* q_len, int shared, int B, int Q,
    int Hq, int Hkv, int D, int page, int num_pages, int max_pages,
    int causal, float scale, dflash_dtype dt, void* out, float* lse, void* ws,
    size_t ws_bytes, dflash_stream_t stream) {
  using namespace dflash;
  if (!(q && k_codes && v_codes && k_scale && v_scale && page_table &&
        kv_len && out && ws))
    return DFLASH_ERR_INVALID_ARG;
  if (dt != DFLASH_BF16 && dt != DFLASH_FP32) return DFLASH_ERR_INVALID_ARG;
  if (!cache_sizes_ok(B, Q, Hq, Hkv, D, page, num_pages, max_pages) ||
      !shared_sizes_ok(B, Q, Hq, Hkv, D))
    return DFLASH_ERR_INVALID_ARG;
  if (shared < 0 || shared % page != 0 || shared / page > max_pages)
    return DFLASH_ERR_INVALID_ARG;
  if (!(scale > -INFINITY && scale < INFINITY)) return DFLASH_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(k_codes, 16) ||
      !aligned_to(v_codes, 16) || !aligned_to(ws, 256))
    return DFLASH_ERR_INVALID_ARG;
  if (ws_bytes < dflash_shared_attn_workspace_bytes(B, Q, Hq, Hkv, D))
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
  a.wait_ns = wait_limit_ns();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      paged_attn_tc_takes(D, dt)
          ? launch_shared_attn_tc(a, shared, sms, ws, s)
      : dt == DFLASH_FP32
          ? launch_simt_d<float>(a, shared, static_cast<float*>(ws), s)
          : launch_simt_d<__nv_bfloat16>(a, shared, static_cast<float*>(ws), s);
  return e == cudaSuccess            ? DFLASH_OK
         : e == cudaErrorNotSupported ? DFLASH_ERR_UNSUPPORTED
                                      : DFLASH_ERR_CUDA;
}

}  // extern "C"
