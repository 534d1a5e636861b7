// The 8-bit paged key/value cache: quantising writes and reads back.
//
// A page holds P tokens of one sequence: codes [pages][Hkv][P][d] and one fp32
// scale per (page, KV head), for K and V apart. A code's value is code * scale.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dil {

enum CacheFmt : int { kFmtE4M3 = 0, kFmtInt8 = 1 };

// The part of a cache's addressing that every kernel needs.
struct CacheGeom {
  const int* table;      // [B][max_pages] page indices
  int B, max_pages;
  int pages, Hkv, lp;    // lp = log2(page size)
  ErrCtx err;
};

// Page of position `pos` of sequence b, or -1 (and the error word raised) when
// the table has no such entry or the entry names no page of the cache.
__device__ __forceinline__ int page_of(const CacheGeom& g, int b, int pos) {
  const int pg = pos >> g.lp;
  int page = -1;
  if (pg < g.max_pages) page = g.table[(size_t)b * g.max_pages + pg];
  if ((unsigned)page >= (unsigned)g.pages) {
    g.err.raise(kErrBadPage);
    return -1;
  }
  return page;
}

// ---------------------------------------------------------------------------
// Code conversions. Scales are powers of two, so x * (1 / scale) and
// code * scale are exact and each code is one rounding (to nearest, ties to
// even) of the value; read back as bf16, which has more fraction bits than
// either format, a value is exact.
// ---------------------------------------------------------------------------
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (FMT == kFmtE4M3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  } else {
    const int ia = max(-127, min(127, __float2int_rn(a))), ib = max(-127, min(127, __float2int_rn(b)));
    const int ic = max(-127, min(127, __float2int_rn(c))), id = max(-127, min(127, __float2int_rn(d)));
    return __byte_perm(__byte_perm(ia, ib, 0x0040), __byte_perm(ic, id, 0x0040), 0x5410);
  }
}

template <int FMT>
__device__ __forceinline__ void decode4(uint32_t x, float (&o)[4]) {
  if constexpr (FMT == kFmtE4M3) {
    const float2 lo = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x & 0xffffu), __NV_E4M3)));
    const float2 hi = __half22float2(
        __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(x >> 16), __NV_E4M3)));
    o[0] = lo.x, o[1] = lo.y, o[2] = hi.x, o[3] = hi.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (float)(int8_t)(x >> (8 * i));
  }
}

// The least power of two 2^e, e >= -126, with amax <= M 2^e for the format's
// largest number M: 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6. amax is given as
// the bits of a finite non-negative float: its exponent is x, and e = x - 8
// (x - 6), one more when the fraction is above M's.
template <int FMT>
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  constexpr int kTopExp = FMT == kFmtE4M3 ? 8 : 6;
  constexpr uint32_t kTopFrac = FMT == kFmtE4M3 ? 0x600000u : 0x7e0000u;
  int e = (int)(amax_bits >> 23) - 127 - kTopExp + ((amax_bits & 0x7fffffu) > kTopFrac ? 1 : 0);
  e = max(e, -126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

struct CacheTokens {
  const int* offsets;  // [B + 1], or null: one token per sequence
  const int* start;    // [B] position of each sequence's first token
  int T;
};

// Tokens of sequence b in the ragged batch, cut to the T rows there are.
__device__ __forceinline__ void token_range(const CacheTokens& t, int b, int& lo, int& n) {
  int a = b, e = b + 1;
  if (t.offsets != nullptr) {
    a = t.offsets[b];
    e = t.offsets[b + 1];
  }
  a = min(max(a, 0), t.T);
  e = min(max(e, a), t.T);
  lo = a;
  n = e - a;
}

struct CacheWriteParams {
  CacheGeom geom;
  CacheTokens tok;
  const __nv_bfloat16* x[2];  // K and V rows [T][Hkv][d], token strides below
  long long stride[2];
  uint8_t* codes[2];
  float* scale[2];
};

// One block per (touched page, KV head, K or V): the page's new rows, its
// scale and, when that grows, the codes already there. A sequence of n tokens
// touches at most floor(n / P) + 2 pages, so sequence b owns the page slots
// from floor(offset_b / P) + 2 b up to the next sequence's first.
template <int D, int FMT>
__global__ void __launch_bounds__(128) cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
  __shared__ int s_seq;
  __shared__ uint32_t s_amax[4];
  const int tid = threadIdx.x, h = blockIdx.y, z = blockIdx.z;
  const int P = 1 << p.geom.lp;
  if (tid == 0) s_seq = -1;
  __syncthreads();
  for (int b = tid; b < p.geom.B; b += 128) {
    int lo, n;
    token_range(p.tok, b, lo, n);
    const long long first = (lo >> p.geom.lp) + 2ll * b;
    const long long last = ((lo + n) >> p.geom.lp) + 2ll * b + 2;
    if (first <= (long long)blockIdx.x && (long long)blockIdx.x < last) s_seq = b;
  }
  __syncthreads();
  const int b = s_seq;
  if (b < 0) return;
  int off, n;
  token_range(p.tok, b, off, n);
  const int start = p.tok.start[b];
  if (n == 0) return;
  if (start < 0 || start > 0x7fffffff - n) {
    p.geom.err.raise(kErrBadPage);
    return;
  }
  const int pg = (start >> p.geom.lp) + (int)((long long)blockIdx.x - (off >> p.geom.lp) - 2ll * b);
  const long long row0 = (long long)pg << p.geom.lp;
  const int lo = (int)max((long long)start, row0), hi = (int)min((long long)start + n, row0 + P);
  if (lo >= hi) return;
  const int page = page_of(p.geom, b, lo);
  if (page < 0) return;

  const __nv_bfloat16* x = p.x[z] + (long long)(off + lo - start) * p.stride[z] + (long long)h * D;
  uint8_t* codes = p.codes[z] + (((size_t)page * p.geom.Hkv + h) << p.geom.lp) * D;
  float* scale = p.scale[z] + (size_t)page * p.geom.Hkv + h;
  constexpr int V = D / 8;  // 16-byte pieces of a row
  const int pieces = (hi - lo) * V;
  // bf16 magnitudes compare as integers; infinities and NaN are 0x7f80 and above
  uint32_t amax = 0;
  for (int i = tid; i < pieces; i += 128) {
    const uint4 u = *reinterpret_cast<const uint4*>(x + (long long)(i / V) * p.stride[z] + (i % V) * 8);
    amax = max(max(amax, u.x & 0x7fffu), (u.x >> 16) & 0x7fffu);
    amax = max(max(amax, u.y & 0x7fffu), (u.y >> 16) & 0x7fffu);
    amax = max(max(amax, u.z & 0x7fffu), (u.z >> 16) & 0x7fffu);
    amax = max(max(amax, u.w & 0x7fffu), (u.w >> 16) & 0x7fffu);
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((tid & 31) == 0) s_amax[tid >> 5] = amax;
  const bool fresh = lo == row0;
  const float was = fresh ? 0.f : *scale;
  __syncthreads();
  amax = max(max(s_amax[0], s_amax[1]), max(s_amax[2], s_amax[3]));
  const bool poisoned = amax >= 0x7f80u || was != was;
  float now = poisoned ? __uint_as_float(0x7fffffffu) : fmaxf(block_scale<FMT>(amax << 16), was);
  const float inv = poisoned ? 0.f : 1.f / now;
  if (!fresh && now > was) {
    const float ratio = was * inv;
    for (int i = tid; i < P * (D / 4); i += 128) {
      const int row = i / (D / 4);
      if (row >= lo - row0 && row < hi - row0) continue;
      uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
      float f[4];
      decode4<FMT>(*w, f);
      *w = encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
    }
  }
  for (int i = tid; i < pieces; i += 128) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (!poisoned)
      u = *reinterpret_cast<const uint4*>(x + (long long)(i / V) * p.stride[z] + (i % V) * 8);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16) * inv;
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * inv;
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(lo - row0 + i / V) * D + (i % V) * 8) =
        make_uint2(encode4<FMT>(f[0], f[1], f[2], f[3]), encode4<FMT>(f[4], f[5], f[6], f[7]));
  }
  if (tid == 0) *scale = now;
}

struct CacheReadParams {
  CacheGeom geom;
  CacheTokens tok;
  __nv_bfloat16* x[2];
  long long stride[2];
  const uint8_t* codes[2];
  const float* scale[2];
};

// One thread per 16 codes of a token and KV head.
template <int D, int FMT>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheReadParams p) {
  constexpr int V = D / 16;
  const long long per = (long long)p.geom.Hkv * V;
  const long long total = per * p.tok.T;
  const int z = blockIdx.z;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const int tok = (int)(i / per), rest = (int)(i % per);
    const int h = rest / V, c = rest % V;
    // last sequence whose first token is at or before tok
    int b = tok;
    if (p.tok.offsets != nullptr) {
      int a = 0, e = p.geom.B;
      while (e - a > 1) {
        const int m = (a + e) >> 1;
        if (p.tok.offsets[m] <= tok) a = m; else e = m;
      }
      b = a;
    }
    if (b >= p.geom.B) continue;
    int off, n;
    token_range(p.tok, b, off, n);
    if (tok < off || tok >= off + n) continue;
    const long long pos = (long long)p.tok.start[b] + tok - off;
    int page = -1;
    if (pos >= 0 && pos <= 0x7fffffff) page = page_of(p.geom, b, (int)pos);
    else p.geom.err.raise(kErrBadPage);
    uint4 u = make_uint4(0, 0, 0, 0);
    float s = 0.f;
    if (page >= 0) {
      const size_t blk = (size_t)page * p.geom.Hkv + h;
      const size_t row = (blk << p.geom.lp) + (pos & ((1 << p.geom.lp) - 1));
      u = *reinterpret_cast<const uint4*>(p.codes[z] + row * D + c * 16);
      s = p.scale[z][blk];
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      decode4<FMT>(w[j], f);
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0] * s, f[1] * s);
      const __nv_bfloat162 e = __floats2bfloat162_rn(f[2] * s, f[3] * s);
      o[2 * j] = *reinterpret_cast<const uint32_t*>(&a);
      o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&e);
    }
    uint4* dst = reinterpret_cast<uint4*>(p.x[z] + (long long)tok * p.stride[z] + h * D + c * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace dil
