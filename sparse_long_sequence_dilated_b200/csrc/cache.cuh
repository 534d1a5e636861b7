// The 8-bit paged key/value cache: quantising writes and reads back.
//
// A page holds P tokens of one sequence: codes [pages][Hkv][P][d] and one fp32
// scale per (page, KV head), for K and V apart. A code's value is code * scale.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace dil {

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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

// The tokens of a page slot: rows r0 .. r0 + rows - 1 of `page`, from token
// `tok` on; rows = 0 when the slot has none. The same in all lanes of a warp.
// A sequence of n tokens touches at most floor(n / P) + 2 pages: sequence b, whose
// first token is off, owns the slots from floor(off / P) + 2 b up to the next one's.
// page = -1 (and the error word raised) for a position or page that there is not.
struct PageRows {
  int page, r0, rows, tok;
};
__device__ __forceinline__ PageRows page_rows(const CacheGeom& g, const CacheTokens& t, long long slot) {
  const int lane = threadIdx.x & 31, P = 1 << g.lp;
  PageRows pr{-1, 0, 0, 0};
  int b = 0, off, n, start;
  if (t.offsets != nullptr) {
    // the slot's sequence: the last one whose first slot is at or before it
    for (int span = g.B;;) {
      const int step = (span + 31) / 32, at = b + lane * step;
      int lo = 0, len = 0, st = 0;
      if (lane * step < span) {
        token_range(t, at, lo, len);
        if (step == 1) st = t.start[at];
      }
      const bool in = lane * step < span && (lo >> g.lp) + 2ll * at <= slot;
      const int k = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0);
      b += k * step;
      if (step == 1) {
        off = __shfl_sync(0xffffffffu, lo, k);
        n = __shfl_sync(0xffffffffu, len, k);
        start = __shfl_sync(0xffffffffu, st, k);
        break;
      }
      span = min(step, span - k * step);
    }
  } else {
    b = (int)min(slot, (long long)g.B - 1);
    token_range(t, b, off, n);
    start = t.start[b];
  }
  const long long skip = slot - (t.offsets != nullptr ? (off >> g.lp) + 2ll * b : b);
  const long long row0 = ((long long)(start >> g.lp) + skip) * P;  // below 0 as a whole, or not at all
  const long long lo = max((long long)start, row0), hi = min((long long)start + n, row0 + P);
  if (n == 0 || lo >= hi) return pr;
  if (lo >= 0 && lo <= 0x7fffffff) pr.page = page_of(g, b, (int)lo);
  else g.err.raise(kErrBadPage);
  pr.r0 = (int)(lo - row0);
  pr.rows = (int)(hi - lo);
  pr.tok = off + (int)(lo - start);
  return pr;
}

struct CacheWriteParams {
  CacheGeom geom;
  CacheTokens tok;
  const __nv_bfloat16* x[2];  // K and V rows [T][Hkv][d], token strides below
  long long stride[2];
  uint8_t* codes[2];
  float* scale[2];
  uint32_t h_mul;             // reciprocal of Hkv (divisor_magic)
  int h_sh;
};

// Largest magnitude of eight bf16 numbers, as their bits compare: infinities and NaN are 0x7f80 and above.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, const uint4& u) {
  m = max(max(m, u.x & 0x7fffu), (u.x >> 16) & 0x7fffu);
  m = max(max(m, u.y & 0x7fffu), (u.y >> 16) & 0x7fffu);
  m = max(max(m, u.z & 0x7fffu), (u.z >> 16) & 0x7fffu);
  return max(max(m, u.w & 0x7fffu), (u.w >> 16) & 0x7fffu);
}
template <int FMT>
__device__ __forceinline__ uint32_t encode_bf16x4(uint32_t a, uint32_t b, float inv) {
  return encode4<FMT>(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                      __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xffff0000u) * inv);
}

// The scale of a page and head after rows of this largest magnitude come to one
// that held `was` (0: the page starts afresh); NaN for numbers that no code holds.
template <int FMT>
__device__ __forceinline__ float next_scale(uint32_t amax, float was) {
  return amax >= 0x7f80u || was != was ? __uint_as_float(0x7fffffffu) : fmaxf(block_scale<FMT>(amax << 16), was);
}

// Rounds a page and head's codes again, rows r0 .. r1 - 1 aside, by `threads` threads from `tid` on.
template <int D, int FMT>
__device__ __forceinline__ void rescale_rows(uint8_t* codes, int P, int r0, int r1, float ratio, int tid, int threads) {
  for (int i = tid; i < P * (D / 16); i += threads) {
    const int row = i / (D / 16);
    if (row >= r0 && row < r1) continue;
    uint4* at = reinterpret_cast<uint4*>(codes) + i;
    const uint4 u = *at;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[4];
      decode4<FMT>(w[k], f);
      o[k] = encode4<FMT>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
    }
    *at = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Bound by loads that follow one another: the offsets (two rounds of the search above
// 32 sequences), the page, then its rows and scale together.
// Few tokens of each sequence: a warp for each (touched page, KV head, K or V).
// A page's first four new rows stay in registers, others are read twice.
template <int D, int FMT>
__global__ void __launch_bounds__(256) cache_append_kernel(const __grid_constant__ CacheWriteParams p) {
  constexpr int C = D / 64;  // 32-bit words of two numbers that a lane has of a row
  constexpr int KEEP = 4;
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
  const uint32_t sz = udiv(unit, p.h_mul, p.h_sh);
  const int h = (int)(unit - sz * (uint32_t)p.geom.Hkv);
  const int z = (int)sz & 1;
  grid_dependency_wait();
  grid_dependency_release();
  const PageRows pr = page_rows(p.geom, p.tok, sz >> 1);
  if (pr.rows == 0 || pr.page < 0) return;
  const __nv_bfloat16* x = p.x[z] + (long long)pr.tok * p.stride[z] + (long long)h * D;
  const size_t blk = (size_t)pr.page * p.geom.Hkv + h;
  uint8_t* codes = p.codes[z] + (blk << p.geom.lp) * D;
  float* scale = p.scale[z] + blk;
  auto load = [&](int i, uint32_t (&u)[C]) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(x + (long long)i * p.stride[z]);
    if constexpr (C == 2) {
      const uint2 v = reinterpret_cast<const uint2*>(src)[lane];
      u[0] = v.x, u[1] = v.y;
    } else {
      u[0] = src[lane];
    }
  };
  const float was = pr.r0 == 0 ? 0.f : *scale;
  uint32_t kept[KEEP][C], amax = 0;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
#pragma unroll
    for (int k = 0; k < C; ++k) kept[i][k] = 0;
    if (i < pr.rows) load(i, kept[i]);
  }
  auto take = [&](const uint32_t (&u)[C]) {
#pragma unroll
    for (int k = 0; k < C; ++k) amax = max(max(amax, u[k] & 0x7fffu), (u[k] >> 16) & 0x7fffu);
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i) take(kept[i]);
  for (int i = KEEP; i < pr.rows; ++i) {
    uint32_t u[C];
    load(i, u);
    take(u);
  }
  const float now = next_scale<FMT>(__reduce_max_sync(0xffffffffu, amax), was);
  const bool poisoned = now != now;
  const float inv = poisoned ? 0.f : 1.f / now;
  if (pr.r0 > 0 && now > was) rescale_rows<D, FMT>(codes, 1 << p.geom.lp, pr.r0, pr.r0 + pr.rows, was * inv, lane, 32);
  auto store = [&](int i, uint32_t (&u)[C]) {
    if (poisoned)
#pragma unroll
      for (int k = 0; k < C; ++k) u[k] = 0;
    uint8_t* dst = codes + (size_t)(pr.r0 + i) * D;
    if constexpr (C == 2) reinterpret_cast<uint32_t*>(dst)[lane] = encode_bf16x4<FMT>(u[0], u[1], inv);
    else reinterpret_cast<uint16_t*>(dst)[lane] = (uint16_t)encode_bf16x4<FMT>(u[0], 0u, inv);
  };
#pragma unroll
  for (int i = 0; i < KEEP; ++i)
    if (i < pr.rows) store(i, kept[i]);
  for (int i = KEEP; i < pr.rows; ++i) {
    uint32_t u[C];
    load(i, u);
    store(i, u);
  }
  if (lane == 0) *scale = now;
}

// Bound by DRAM: two bytes in and one out a number. 131072 tokens of 32 heads,
// d = 128 (3.2 GB) take 527 us as a call among others (6.1 TB/s), and 490 to 498
// replayed from a graph over inputs that lie in place (6.5 TB/s), where the page as
// the fastest index instead of the head, and rows read twice, took 650 us.
//
// Ragged stretches: W warps for each (touched page, KV head), K and then V, with
// all of its new rows in registers, N times 16 numbers a lane, so that they are read once.
// Heads are the fastest index: blocks that run together read whole rows.
// Four blocks on an SM (64 registers), three for the largest units, whose loads need
// no more: 199 to 178 us and 81 to 74 us for small pages, 472 to 463 for 128-token ones.
template <int D, int FMT, int W, int N>
__global__ void __launch_bounds__(256, W == 8 ? 3 : 4) cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
  constexpr int V = D / 16;  // pieces of 16 numbers of a row
  __shared__ uint32_t s_amax[2][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = threadIdx.x % (W * 32);  // in the unit
  const uint32_t unit = blockIdx.x * (8 / W) + warp / W;
  const uint32_t slot = udiv(unit, p.h_mul, p.h_sh);
  const int h = (int)(unit - slot * (uint32_t)p.geom.Hkv);
  const int P = 1 << p.geom.lp;
  grid_dependency_wait();
  grid_dependency_release();
  const PageRows pr = page_rows(p.geom, p.tok, slot);
  const bool work = pr.rows > 0 && pr.page >= 0;
  const int r0 = pr.r0, rows = work ? pr.rows : 0;
  const size_t blk = work ? (size_t)pr.page * p.geom.Hkv + h : 0;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const __nv_bfloat16* x = p.x[z] + (long long)pr.tok * p.stride[z] + (long long)h * D;
    uint8_t* codes = p.codes[z] + (blk << p.geom.lp) * D;
    float* scale = p.scale[z] + blk;
    uint4 u[N][2];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = tid + i * W * 32;
      u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
      if (k / V < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + (long long)(k / V) * p.stride[z] + (k % V) * 16);
        u[i][0] = src[0], u[i][1] = src[1];
      }
    }
    const float was = work && r0 > 0 ? *scale : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = max_magnitude(max_magnitude(amax, u[i][0]), u[i][1]);
    amax = __reduce_max_sync(0xffffffffu, amax);
    if constexpr (W > 1) {
      if (lane == 0) s_amax[z][warp] = amax;
      __syncthreads();
      const int first = warp / W * W;
#pragma unroll
      for (int i = 0; i < W; ++i) amax = max(amax, s_amax[z][first + i]);
    }
    if (!work) continue;
    const float now = next_scale<FMT>(amax, was);
    const bool poisoned = now != now;
    const float inv = poisoned ? 0.f : 1.f / now;
    if (r0 > 0 && now > was) rescale_rows<D, FMT>(codes, P, r0, r0 + rows, was * inv, tid, W * 32);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = tid + i * W * 32;
      if (k / V >= rows) continue;
      if (poisoned) u[i][0] = u[i][1] = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(codes + (size_t)r0 * D + (size_t)k * 16) =
          make_uint4(encode_bf16x4<FMT>(u[i][0].x, u[i][0].y, inv), encode_bf16x4<FMT>(u[i][0].z, u[i][0].w, inv),
                     encode_bf16x4<FMT>(u[i][1].x, u[i][1].y, inv), encode_bf16x4<FMT>(u[i][1].z, u[i][1].w, inv));
    }
    if (tid == 0) *scale = now;
  }
}

struct CacheReadParams {
  CacheGeom geom;
  CacheTokens tok;
  __nv_bfloat16* x[2];
  long long stride[2];
  const uint8_t* codes[2];
  const float* scale[2];
  int pieces;                 // of 16 codes that a token has
  uint32_t p_mul;             // reciprocal of pieces (divisor_magic)
  int p_sh;
};

constexpr int kReadThreads = 256;

// The last sequence whose first token is at or before tok. One warp.
__device__ __forceinline__ int sequence_of(const CacheReadParams& p, long long tok) {
  int b = 0;
  for (int span = p.geom.B; span > 1;) {
    const int lane = threadIdx.x & 31, step = (span + 31) / 32, at = b + lane * step;
    const bool in = lane * step < span && p.tok.offsets[at] <= tok;
    const int k = max(__popc(__ballot_sync(0xffffffffu, in)) - 1, 0);
    b += k * step;
    span = min(step, span - k * step);
  }
  return b;
}

// Bound by DRAM: one byte in and two out a number (131072 tokens of 32 heads, d = 128:
// 538 to 547 us as a call among others, 5.9 to 6.0 TB/s; 505 to 517 replayed from a
// graph). Page by page, as writes go, the rows would go out in pieces of 256 bytes:
// 583 us where this took 507.
//
// A block has kReadThreads * EACH successive pieces of 16 codes, in the order of the rows that
// it writes: they are two thirds of the traffic. Two warps find the sequences of its first and
// its last token; a thread's own lies between them.
template <int D, int FMT, int EACH>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheReadParams p) {
  constexpr int V = D / 16;
  __shared__ int s_seq[2];
  const int tid = threadIdx.x, warp = tid >> 5, z = blockIdx.y;
  const long long first = (long long)blockIdx.x * (kReadThreads * EACH);
  const long long tok0 = first / p.pieces;
  const uint32_t skip = (uint32_t)(first - tok0 * p.pieces);
  grid_dependency_wait();
  grid_dependency_release();
  if (p.tok.offsets != nullptr) {
    if (warp < 2) {
      const long long last = min(tok0 + udiv(skip + kReadThreads * EACH - 1, p.p_mul, p.p_sh), (long long)p.tok.T - 1);
      const int b = sequence_of(p, warp == 0 ? tok0 : last);
      if ((tid & 31) == 0) s_seq[warp] = b;
    }
    __syncthreads();
  }
  long long tok[EACH], row[EACH];  // row < 0: reads as zeros
  size_t blk[EACH];
  uint32_t piece[EACH];
  bool real[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const uint32_t j = skip + tid + i * kReadThreads, dt = udiv(j, p.p_mul, p.p_sh);
    tok[i] = tok0 + dt;
    piece[i] = j - dt * (uint32_t)p.pieces;
    real[i] = tok[i] < p.tok.T;
    row[i] = -1;
    blk[i] = 0;
    if (!real[i]) continue;
    int b = (int)tok[i];
    if (p.tok.offsets != nullptr) {
      b = s_seq[0];
      for (int e = s_seq[1] + 1; e - b > 1;) {
        const int m = (b + e) >> 1;
        if (p.tok.offsets[m] <= tok[i]) b = m; else e = m;
      }
    }
    int off, n;
    token_range(p.tok, b, off, n);
    real[i] = b < p.geom.B && tok[i] >= off && tok[i] < off + n;
    if (!real[i]) continue;
    const long long pos = (long long)p.tok.start[b] + tok[i] - off;
    int page = -1;
    if (pos >= 0 && pos <= 0x7fffffff) page = page_of(p.geom, b, (int)pos);
    else p.geom.err.raise(kErrBadPage);
    if (page >= 0) {
      blk[i] = (size_t)page * p.geom.Hkv + piece[i] / V;
      row[i] = (long long)((blk[i] << p.geom.lp) + (size_t)(pos & ((1 << p.geom.lp) - 1)));
    }
  }
  uint4 u[EACH];
  float sc[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    u[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0.f;
    if (row[i] >= 0) {
      u[i] = *reinterpret_cast<const uint4*>(p.codes[z] + (size_t)row[i] * D + (piece[i] % V) * 16);
      sc[i] = p.scale[z][blk[i]];
    }
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (!real[i]) continue;
    const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[4];
      decode4<FMT>(w[j], f);
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0] * sc[i], f[1] * sc[i]);
      const __nv_bfloat162 e = __floats2bfloat162_rn(f[2] * sc[i], f[3] * sc[i]);
      o[2 * j] = *reinterpret_cast<const uint32_t*>(&a);
      o[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&e);
    }
    uint4* dst = reinterpret_cast<uint4*>(p.x[z] + tok[i] * p.stride[z] + (long long)piece[i] * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace dil
