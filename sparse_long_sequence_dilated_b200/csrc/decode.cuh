// Dilated attention of single query tokens over the 8-bit paged cache.
//
// A token at position t takes part in pattern (w, r) for the heads h with
// h mod r = (t - s) mod r, s = floor(t / w) w its segment's start; those heads
// then all attend the same rows: t, t - r, t - 2 r, ... down to s. The output is
// one softmax over the multiset union of the patterns' rows.
#pragma once

#include "cache.cuh"

namespace dil {

struct DecodeParams {
  CacheGeom geom;
  const __nv_bfloat16* q;  // [T][H][d], token stride below
  long long q_stride;
  const uint8_t* codes[2];
  const float* scale[2];
  const int* seq;  // [T] sequence of each token, or null: token i is sequence i's
  const int* pos;  // [T]
  __nv_bfloat16* out;
  float* lse;
  int T, H;
  float qk_scale;  // log2(e) / sqrt(d)
  int npat;
  int w[kMaxPat], r[kMaxPat];
};

// One block per (token, query head); each warp takes every fourth row of every
// pattern and keeps its own running maximum and sum.
template <int D, int FMT>
__global__ void __launch_bounds__(128) decode_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int C = D / 32;
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const int t = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = h / (p.H / p.geom.Hkv);
  const int b = p.seq != nullptr ? p.seq[t] : t;
  int pos = p.pos[t];
  if (pos >= 0 && ((unsigned)b >= (unsigned)p.geom.B || (pos >> p.geom.lp) >= p.geom.max_pages)) {
    p.geom.err.raise(kErrBadPage);
    pos = -1;
  }
  float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    q[i] = __bfloat162float(p.q[t * p.q_stride + h * D + lane * C + i]) * p.qk_scale;
    o[i] = 0.f;
  }
  if (pos >= 0) {
    for (int j = 0; j < p.npat; ++j) {
      const int start = pos / p.w[j] * p.w[j], off = (pos - start) % p.r[j];
      if (h % p.r[j] != off) continue;
      const int n = (pos - start) / p.r[j] + 1;
      for (int k = warp; k < n; k += 4) {
        const int x = pos - k * p.r[j];
        const int page = page_of(p.geom, b, x);
        if (page < 0) continue;
        const size_t blk = (size_t)page * p.geom.Hkv + hk;
        const size_t row = (blk << p.geom.lp) + (x & ((1 << p.geom.lp) - 1));
        float kk[4], vv[4], dot = 0.f;
        if constexpr (C == 4) {
          decode4<FMT>(*reinterpret_cast<const uint32_t*>(p.codes[0] + row * D + lane * 4), kk);
          decode4<FMT>(*reinterpret_cast<const uint32_t*>(p.codes[1] + row * D + lane * 4), vv);
        } else {
          decode4<FMT>(*reinterpret_cast<const uint16_t*>(p.codes[0] + row * D + lane * 2), kk);
          decode4<FMT>(*reinterpret_cast<const uint16_t*>(p.codes[1] + row * D + lane * 2), vv);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) dot += q[i] * kk[i];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        dot *= p.scale[0][blk];
        const float mn = fmaxf(m, dot);
        const float c = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(dot - mn);
        const float sv = p.scale[1][blk];
        l = l * c + e;
#pragma unroll
        for (int i = 0; i < C; ++i) o[i] = o[i] * c + e * (vv[i] * sv);
        m = mn;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) s_o[warp][lane * C + i] = o[i];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  float mx = -INFINITY, sum = 0.f;
  for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s_m[i]);
  float wgt[4];
  for (int i = 0; i < 4; ++i) {
    wgt[i] = s_m[i] == -INFINITY ? 0.f : exp2f(s_m[i] - mx);
    sum += s_l[i] == 0.f ? 0.f : s_l[i] * wgt[i];
  }
  const size_t oi = (size_t)t * p.H + h;
  for (int i = threadIdx.x; i < D; i += 128) {
    float a = 0.f;
    for (int k = 0; k < 4; ++k) a += s_l[k] == 0.f ? 0.f : s_o[k][i] * wgt[k];
    p.out[oi * D + i] = __float2bfloat16(sum == 0.f ? 0.f : a / sum);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[oi] = sum == 0.f ? -INFINITY : 0.69314718055994531f * (mx + log2f(sum));
}

}  // namespace dil
