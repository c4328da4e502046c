// Attention over the paged 8-bit cache on the CUDA cores (fp32 storage, or heads
// wider than the tensor-core kernels take): the kernel and the one that joins
// its parts.
//
// Mathematics.  s_t = scale <q, k_t>; out = sum_t p_t v_t / l with
// p_t = exp(s_t - m), l = sum_t p_t, one pass over the tokens with the
// running maximum m (accumulators are multiplied by exp(m_old - m_new)).
// Two parts of a sequence with (m1, l1, o1), (m2, l2, o2) join as
// o = sum_i exp(m_i - m) o_i, l likewise, so a long sequence is cut into
// parts that run at the same time.
//
// A row is a (query, head) pair; the Hq / Hkv heads that share a key head
// read its tokens together.  The CUDA-core kernel takes up to eight rows of
// one key head and a part of the tokens; its warps take tiles of 32 tokens
// in turn, each with sums of its own (joined in shared memory at the end),
// so that few rows still make many independent warps.  For the scores
// lane = token, which reads its key's codes 16 at a time (the tile's lines
// are used whole, over the steps); for the sum of values lane = four
// dimensions, one line per token.  No tile passes through shared memory.
//
// What bounds it: the latency of the codes' loads and of each warp's chain of
// fp32 products; 16 warps fit an SM.  fp32, heads of 128: one row of 60000
// tokens and 8 key heads 184 us (123 MB), 60 such rows of 3000 tokens 473 us
// (368 MB); without asking for the next tile's lines 230 us and 605 us.  32 x 9
// queries of 4000 tokens, 36 rows a head: 1.6 ms.
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"

namespace dflash {
namespace {

constexpr int kRows = 8;      // rows of a CTA
constexpr int kTok = 32;      // tokens of a tile
constexpr int kWarps = 8;
constexpr int kMaxSplits = 32;
// Values are added up times 2^-32, exactly: of the largest scale (2^120) some
// hundred would pass fp32's range before they are divided by their weights.
constexpr float kDown = 0x1p-32f, kUp = 0x1p32f;

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

__device__ __forceinline__ void prefetch(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// W = words of four dimensions that a lane holds; with G = 2 the halves of a
// warp take two tokens' values at a time (heads of up to 64 dimensions).
// Two CTAs to an SM (128 registers).  Three (80, some spilt) where heads of 80
// to 128 have full row tiles and sequences are not cut: 32 x 9 queries of 4000
// tokens, 36 rows a head, 1.57 instead of 1.79 ms; cut sequences, four rows and
// narrow heads lose (one row of 60000 tokens 267 instead of 223 us, 60 such
// rows of 3000 683 instead of 605 us, D = 64 150 instead of 126 us).
// kShared: the first view.shared tokens of every sequence are the first one's; the
// grid's first CTAs take them, with the rows of all sequences, the others each
// sequence's own tokens, and the parts of a row are those of both.
struct SharedView {
  int shared;        // tokens, whole pages
  int splits;        // parts that they are cut into
  int row_tiles;     // of all sequences' rows
  unsigned items;    // CTAs that take them
};
template <typename T, int W, int G, int kPerSm, bool kShared = false>
__global__ void __launch_bounds__(kWarps * 32, kPerSm)
    paged_attn_simt_kernel(const __grid_constant__ PagedAttnArgs a, int splits,
                           int row_tiles, float* __restrict__ part,
                           const SharedView view) {
  extern __shared__ float4 smem4[];
  const int D = a.D;
  float* sq = reinterpret_cast<float*>(smem4);  // [kRows][D]
  float* so = sq + kRows * D;                   // [kWarps][kRows][D]
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int item = blockIdx.x;
  const bool prefix = kShared && blockIdx.x < view.items;
  const int cuts = prefix ? view.splits : splits;
  if (kShared && !prefix) item -= view.items;
  const int sp = item % cuts;
  item /= cuts;
  const int tiles = prefix ? view.row_tiles : row_tiles;
  const int tile = item % tiles;
  item /= tiles;
  const int hk = item % a.Hkv, b = item / a.Hkv;
  const int g = a.Hq / a.Hkv;
  const int row0 = tile * kRows;
  const int rows_here = min(kRows, (prefix ? a.B : 1) * a.Q * g - row0);
  // row r of this CTA: its query among all sequences' and its head
  auto query_of = [&](int r) { return b * a.Q + (row0 + r) / g; };
  auto row_of = [&](int r) {
    return (long long)query_of(r) * a.Hq + hk * g + (row0 + r) % g;
  };
  bool bad = false;
  int n = attn_clamp(a.kv_len[b], a.max_pages * (long long)a.page, &bad);
  int nq = attn_clamp(a.q_len ? a.q_len[b] : a.Q, a.Q, &bad);
  if (bad && tid == 0) raise_error(a.err, kErrBadIndex);
  // tokens each row sees: t < lim (none for a row without a query)
  int lim[kRows], most = 0;
  uint32_t live = 0;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    int qi = (row0 + r) / g;
    if (prefix && r < rows_here) {
      const int of = qi / a.Q;
      qi -= of * a.Q;
      n = attn_clamp(a.kv_len[of], a.max_pages * (long long)a.page, &bad);
      nq = attn_clamp(a.q_len ? a.q_len[of] : a.Q, a.Q, &bad);
    }
    lim[r] = r >= rows_here || qi >= nq
                 ? 0
                 : a.causal ? max(0, min(n, n - nq + qi + 1)) : n;
    if (prefix) lim[r] = min(lim[r], view.shared);
    if (r < rows_here && qi < nq) live |= 1u << r;
    most = max(most, lim[r]);
  }
  for (int i = tid; i < kRows * D; i += kWarps * 32) {
    const int r = i / D;
    sq[i] = live >> r & 1 ? to_f32(static_cast<const T*>(
                                a.q)[(size_t)row_of(r) * D + i % D]) *
                                a.scale
                          : 0.f;
  }
  const int from = kShared && !prefix ? view.shared : 0;  // first token
  const int span = max(0, most - from);
  int chunk = (span + cuts - 1) / cuts;
  chunk = max((chunk + kTok - 1) / kTok * kTok, 2 * kTok);
  const int t0 = from + (int)min((long long)sp * chunk, (long long)span);
  const int t1 = (int)min((long long)t0 + chunk, (long long)from + span);
  __syncthreads();

  const int part_lane = G == 2 ? lane & 15 : lane;  // words of a value
  float m[kRows], l[kRows], o[kRows][4 * W];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int d = 0; d < 4 * W; ++d) o[r][d] = 0.f;
  }
  // The page of a lane's token is looked up, and its lines asked for, a tile
  // ahead: they take longer than the tile.
  auto page_of = [&](int t) {
    int id = -1;
    if (t < t1) {
      id = a.table[(size_t)b * a.max_pages + t / a.page];
      if (id < 0 || id >= a.num_pages) {
        raise_error(a.err, kErrBadIndex);
        id = -1;
      }
    }
    return id;
  };
  auto ask = [&](int id, int t) {
    if (id < 0) return;
    const size_t at = (((size_t)id * a.Hkv + hk) * a.page + t % a.page) * D;
    for (int d = 0; d < D; d += 128) {
      prefetch(a.k_codes + at + d);
      prefetch(a.v_codes + at + d);
    }
  };
  const int t_first = t0 + wid * kTok + lane;
  int id = page_of(t_first);
  ask(id, t_first);
  for (int base = t0 + wid * kTok; base < t1; base += kWarps * kTok) {
    // this lane's token: where its codes are, its scales
    const int t = base + lane;
    const int next = page_of(t + kWarps * kTok);
    const size_t ph = id >= 0 ? (size_t)id * a.Hkv + hk : 0;
    const size_t at = (ph * a.page + t % a.page) * D;
    const float ks = id >= 0 ? a.k_scale[ph] : 0.f;
    const float vs = id >= 0 ? a.v_scale[ph] * kDown : 0.f;
    float s[kRows] = {};
#pragma unroll 2
    for (int d = 0; d < D; d += 16) {
      uint4 kc = make_uint4(0, 0, 0, 0);
      if (id >= 0) kc = *reinterpret_cast<const uint4*>(a.k_codes + at + d);
      float k[16];
      decode16(kc, ks, k);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows_here) break;  // uniform
        const float4* q4 = reinterpret_cast<const float4*>(sq + r * D + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 q = q4[i];
          s[r] = fmaf(q.x, k[4 * i], fmaf(q.y, k[4 * i + 1],
                 fmaf(q.z, k[4 * i + 2], fmaf(q.w, k[4 * i + 3], s[r]))));
        }
      }
    }
    ask(next, t + kWarps * kTok);
    float w[kRows];  // this lane's token's weights, times its values' scale
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      w[r] = 0.f;
      if (r >= rows_here) break;
      const float x = t < min(lim[r], t1) ? s[r] : -INFINITY;
      const float mn = fmaxf(m[r], warp_max(x));
      const float f = mn == -INFINITY ? 1.f : expf(m[r] - mn);
      const float p = x == -INFINITY ? 0.f : expf(x - mn);
      l[r] = l[r] * f + p;
      m[r] = mn;
      w[r] = p * vs;
#pragma unroll
      for (int d = 0; d < 4 * W; ++d) o[r][d] *= f;
    }
    const long long mine = id >= 0 ? (long long)at : -1;
#pragma unroll 4
    for (int i = 0; i < kTok; i += G) {
      const int lane_of = G == 2 ? i + (lane >> 4) : i;
      const long long src = __shfl_sync(0xffffffffu, mine, lane_of);
      uint32_t v[W];
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const int d = 4 * (part_lane + 32 * c);
        v[c] = src >= 0 && d < D
                   ? *reinterpret_cast<const uint32_t*>(a.v_codes + src + d)
                   : 0;
      }
      float x[4 * W];
#pragma unroll
      for (int c = 0; c < W; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 f2 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
              (__nv_fp8x2_storage_t)(v[c] >> (16 * j)), __NV_E4M3)));
          x[4 * c + 2 * j] = f2.x;
          x[4 * c + 2 * j + 1] = f2.y;
        }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r >= rows_here) break;
        const float wr = __shfl_sync(0xffffffffu, w[r], lane_of);
#pragma unroll
        for (int d = 0; d < 4 * W; ++d) o[r][d] = fmaf(wr, x[d], o[r][d]);
      }
    }
    id = next;
  }
  // ---- the warps' sums ------------------------------------------------------
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r >= rows_here) break;
    const float sum = warp_sum(l[r]);
    if (lane == 0) {
      s_m[wid][r] = m[r];
      s_l[wid][r] = sum;
    }
#pragma unroll
    for (int d = 0; d < 4 * W; ++d)
      if (G == 2) o[r][d] += __shfl_xor_sync(0xffffffffu, o[r][d], 16);
#pragma unroll
    for (int c = 0; c < W; ++c) {
      const int d = 4 * (part_lane + 32 * c);
      if (d < D && (G == 1 || lane < 16))
        *reinterpret_cast<float4*>(so + ((size_t)wid * kRows + r) * D + d) =
            make_float4(o[r][4 * c], o[r][4 * c + 1], o[r][4 * c + 2],
                        o[r][4 * c + 3]);
    }
  }
  __syncthreads();
  const long long rows = (long long)a.B * a.Q * a.Hq;
  const int slot = kShared && !prefix ? view.splits + sp : sp;
  const int slots = kShared ? view.splits + splits : splits;
  for (int i = tid; i < rows_here * D; i += kWarps * 32) {
    const int r = i / D, d = i % D;
    const long long row = row_of(r);
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) top = fmaxf(top, s_m[v][r]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      const float f = s_m[v][r] == -INFINITY ? 0.f : expf(s_m[v][r] - top);
      sum = fmaf(f, s_l[v][r], sum);
      if (f != 0.f) acc = fmaf(f, so[((size_t)v * kRows + r) * D + d], acc);
    }
    const bool seen = sum > 0.f || sum != sum;  // a NaN stays one
    if (slots == 1) {
      static_cast<T*>(a.out)[row * D + d] =
          from_f32<T>(seen ? acc / sum * kUp : 0.f);
      if (d == 0 && a.lse) a.lse[row] = seen ? top + logf(sum) : -INFINITY;
    } else {
      part[((size_t)slot * rows + row) * D + d] = acc;
      if (d == 0) {
        float* pm = part + (size_t)slots * rows * D +
                    ((size_t)slot * rows + row) * 2;
        pm[0] = top;
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
  const bool seen = l > 0.f || l != l;  // a NaN stays one
  const float inv = seen ? kUp / l : 0.f;
  constexpr int kAt = 8;  // parts on their way at once
  for (int base = 0; base < D; base += 128) {  // whole warps shuffle
    const int d = base + 4 * lane;  // D % 16 == 0
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < splits; s0 += kAt) {
      float4 x[kAt];
      float ws[kAt];
#pragma unroll
      for (int s = 0; s < kAt; ++s) {
        ws[s] = __shfl_sync(0xffffffffu, w, s0 + s);  // 0 past the splits
        x[s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d < D && ws[s] != 0.f)
          x[s] = *reinterpret_cast<const float4*>(
              part + ((size_t)(s0 + s) * rows + row) * D + d);
      }
#pragma unroll
      for (int s = 0; s < kAt; ++s) {
        o.x = fmaf(ws[s], x[s].x, o.x);
        o.y = fmaf(ws[s], x[s].y, o.y);
        o.z = fmaf(ws[s], x[s].z, o.z);
        o.w = fmaf(ws[s], x[s].w, o.w);
      }
    }
    if (d < D) {
      T* to = out + row * D + d;
      to[0] = from_f32<T>(o.x * inv);
      to[1] = from_f32<T>(o.y * inv);
      to[2] = from_f32<T>(o.z * inv);
      to[3] = from_f32<T>(o.w * inv);
    }
  }
  if (lane == 0 && lse) lse[row] = seen ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace dflash
