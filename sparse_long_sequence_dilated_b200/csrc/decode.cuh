// Dilated attention of single query tokens over the 8-bit paged cache.
//
// Which rows. A token at position t takes part in pattern (w, r) for the heads
// h with h mod r = (t - s) mod r, s = floor(t / w) w its segment's start; those
// heads then all attend the same rows: t, t - r, t - 2 r, ... down to s. The
// output is one softmax over the multiset union of the patterns' rows, so a row
// that several patterns hold is read once and weighted by their number.
//
// Items. An item is a (token, KV head) pair with up to 8 (NB = 1) or 16
// (NB = 2) of the query heads that share the KV head: they share its rows too.
// Patterns are sorted by r. A row is walked by the first pattern, for that
// head, that holds it. Where r_l divides r_j and every head of the item that
// takes part in j takes part in l, l walks all of j's rows from s_l on, so j's
// walk ends there; what overlap remains (r that do not divide one another) is
// masked row by row. An item's walks, in tiles of TR rows, are its work.
//
// Split. The tiles of all items form one sequence that is cut into equal
// contiguous ranges, one for each warp of a persistent grid, wherever the cut
// falls: no batch shape, length or head count leaves SMs idle. An item inside
// one range is finished by its warp; warps of a block join theirs in shared
// memory; items cut between blocks leave partials that decode_join_kernel
// combines in block order (no atomics: the same call gives the same bits).
#pragma once

#include "cache.cuh"

namespace dil {

constexpr int kDecWarps = 8;
constexpr int kDecMaxBlocks = 320;  // partial slots in the workspace; two blocks on each of 148 SMs fit
constexpr int kDecGroups = 1024;    // most groups of items that the plan sums

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
  int T, H, G;               // G query heads to a KV head
  int nsub;                  // items that a KV head's query heads make up
  int per_token;             // Hkv * nsub
  uint32_t pt_mul, ns_mul;   // reciprocals of per_token and nsub (divisor_magic)
  int pt_sh, ns_sh;
  int items;
  int group;                 // items whose tile counts a plan block sums
  float qk_scale;            // log2(e) / sqrt(d)
  int npat;                  // patterns, by ascending r
  int w[kMaxPat], r[kMaxPat];
  uint32_t w_mul[kMaxPat], r_mul[kMaxPat];
  int w_sh[kMaxPat], r_sh[kMaxPat];
  uint32_t r_inv[kMaxPat], r_lim[kMaxPat];  // divisibility by r (see divides)
  int r_rot[kMaxPat];
  uint32_t divisors[kMaxPat];               // earlier patterns whose r divides this one's
  // workspace
  int* counts;               // [items] tiles
  long long* sums;           // [kDecGroups] tiles of each group
  int* begun;                // [blocks] item that began before the block's range, or -1
  int* unfinished;           // [blocks] item that begins in the block's range and ends past it, or -1
  float* part;               // [blocks][2] partials of those two
  float* warp_part;          // [blocks][kDecWarps] partials of items that end in a warp's range
  int part_heads, part_stride;  // heads and floats of a partial: sums [heads][D], (m, mv, l, -) [heads]
};

// x mod r == 0, for x < 2^31 and r = 2^rot odd: x times the inverse of odd
// modulo 2^32, rotated right by rot, is x / r when r divides x and more than
// (2^32 - 1) / r otherwise (Granlund and Montgomery 1994, section 9).
__device__ __forceinline__ bool divides(const DecodeParams& p, int i, int x) {
  const uint32_t y = (uint32_t)x * p.r_inv[i];
  return __funnelshift_r(y, y, p.r_rot[i]) <= p.r_lim[i];
}

template <int D_, int NB_>
struct DecodeCfg {
  static constexpr int D = D_, NB = NB_;
  static constexpr int HEADS = 8 * NB;
  static constexpr int TR = D == 128 ? 16 : 32;  // rows of a tile: 4 KB of codes either way
  static constexpr int RB = TR / 16;
  static constexpr int BLOCKS_PER_SM = NB == 1 ? 2 : 1;  // by registers: 16 heads keep 64 sums a thread
  static constexpr int STAGES = NB == 1 ? 3 : 6;
  static constexpr int STAGE_BYTES = 2 * TR * D + 2 * TR * 4;
  static constexpr int RING_BYTES = kDecWarps * STAGES * STAGE_BYTES;
  static constexpr int STATS = kDecWarps * 2 * HEADS;  // float4 each
  static constexpr int SMEM_BYTES = RING_BYTES + STATS * 16 + kDecWarps * 3 * 4;
  static_assert(kDecGroups * 8 + 64 <= RING_BYTES, "the group sums share the ring's memory");
  static_assert(HEADS * D * 4 <= STAGES * STAGE_BYTES, "a warp's partial fits in its ring");
};

// What a warp knows of an item. Lane j holds pattern j's walk: rows
// base + k r_j, k < n, in the item's tiles up to `tend`; s is its segment's start
// and heads the item's heads (bits) that take part.
struct DecodeItem {
  int token, b, pos, hk, h0, nh;
  int tiles;
  int s, base, n, tend;
  uint32_t heads;
};

template <int TR, int HEADS>
__device__ __forceinline__ void load_item(const DecodeParams& p, int item, DecodeItem& it) {
  const int lane = threadIdx.x & 31;
  it.token = (int)udiv((uint32_t)item, p.pt_mul, p.pt_sh);
  const int c = item - it.token * p.per_token;
  it.hk = (int)udiv((uint32_t)c, p.ns_mul, p.ns_sh);
  const int first = (c - it.hk * p.nsub) * HEADS;
  it.h0 = it.hk * p.G + first;
  it.nh = min(HEADS, p.G - first);
  it.b = p.seq != nullptr ? p.seq[it.token] : it.token;
  it.pos = p.pos[it.token];
  if (it.pos >= 0 &&
      ((unsigned)it.b >= (unsigned)p.geom.B || (it.pos >> p.geom.lp) >= p.geom.max_pages)) {
    p.geom.err.raise(kErrBadPage);
    it.pos = -1;
  }
  it.heads = 0;
  it.n = 0;
  it.s = 0;
  it.base = 0;
  if (lane < p.npat && it.pos >= 0) {
    const int w = p.w[lane], r = p.r[lane];
    const uint32_t rm = p.r_mul[lane];
    const int rs = p.r_sh[lane];
    it.s = (int)udiv((uint32_t)it.pos, p.w_mul[lane], p.w_sh[lane]) * w;
    const int rel = it.pos - it.s;
    const int steps = (int)udiv((uint32_t)rel, rm, rs);
    const int off = rel - steps * r;
    it.base = it.s + off;
    it.n = steps + 1;
    const int first_k = off - (it.h0 - (int)udiv((uint32_t)it.h0, rm, rs) * r);
    for (uint32_t k = first_k < 0 ? first_k + r : first_k; k < (uint32_t)it.nh; k += (uint32_t)r)
      it.heads |= 1u << k;  // k + r stays below 2^32
  }
  const uint32_t div = lane < p.npat ? p.divisors[lane] : 0u;
  int limit = 0x7fffffff;
  for (int l = 0; l + 1 < p.npat; ++l) {
    const int sl = __shfl_sync(0xffffffffu, it.s, l);
    const uint32_t hl = __shfl_sync(0xffffffffu, it.heads, l);
    if ((div >> l & 1u) && (it.heads & ~hl) == 0) limit = min(limit, sl);
  }
  if (it.heads == 0) {
    it.n = 0;
  } else if (limit <= it.pos) {
    it.n = limit > it.base
               ? (int)udiv((uint32_t)(limit - 1 - it.base), p.r_mul[lane], p.r_sh[lane]) + 1
               : 0;
  }
  it.tend = (int)(((uint32_t)it.n + TR - 1) / TR);
#pragma unroll
  for (int s = 1; s < kMaxPat; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, it.tend, s);
    if (lane >= s) it.tend += v;
  }
  // an item without rows keeps one empty tile: the warp that has it writes its zeros
  it.tiles = max(1, __shfl_sync(0xffffffffu, it.tend, p.npat - 1));
}

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// D += A B, A 16 x 16 and B 16 x 8 fp16, D fp32.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_release() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Plan: the tile count of every item and of every group of items.
// ---------------------------------------------------------------------------
template <int TR, int HEADS>
__global__ void __launch_bounds__(kDecWarps * 32)
    decode_plan_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ long long s_sum[kDecWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_release();
  const long long first = (long long)blockIdx.x * p.group;
  const int end = (int)min(first + p.group, (long long)p.items);
  long long sum = 0;
  for (int i = (int)first + warp; i < end; i += kDecWarps) {
    DecodeItem it;
    load_item<TR, HEADS>(p, i, it);
    if (lane == 0) p.counts[i] = it.tiles;
    sum += it.tiles;
  }
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0;
    for (int i = 0; i < kDecWarps; ++i) sum += s_sum[i];
    p.sums[blockIdx.x] = sum;
  }
}

// The fp16 values (exact) of the low and high two codes of x.
template <int FMT>
__device__ __forceinline__ void codes_to_half(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kFmtE4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  } else {
    // 0x6400 | u is 1024 + u in fp16; u = code + 128
    const uint32_t u = x ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
    const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ra);
    hi = *reinterpret_cast<const uint32_t*>(&rb);
  }
}

// A maximum below every score, for heads that have seen no row: differences
// with it stay finite.
constexpr float kNoMax = -3e38f;
// Maxima are raised only when a score exceeds them by more than this (log2):
// probabilities then reach 2^4, times at most 16 patterns; kPBias lifts them
// to 2^15, within fp16, so that the smallest that fp16 keeps is 2^-32 of the largest.
constexpr float kMaxSlack = 4.f;
constexpr float kPBias = 7.f;

// Final value of one output element and its head's statistics.
__device__ __forceinline__ float final_factor(float m, float mv, float l) {
  return l == 0.f ? 0.f : exp2f(mv - m - kPBias) / l;
}
__device__ __forceinline__ float final_lse(float m, float l) {
  return l == 0.f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
}

// Partials: sums [heads][D], then (m, mv, l, unused) of each head.
// Combines an item's partials of warps from .. last (last: the head that ends
// it, when `ended`) into the result, or into dst.
template <int D, int NB>
__device__ void join_warps(const DecodeParams& p, int item, int from, int last, bool ended,
                           const int* s_tail, const float4* s_stat, const uint8_t* smem,
                           const float* warp_part, float* dst) {
  using Cfg = DecodeCfg<D, NB>;
  constexpr int HEADS = Cfg::HEADS;
  const int token = item / p.per_token, c = item % p.per_token;
  const int hk = c / p.nsub, first = (c % p.nsub) * HEADS;
  const int nh = min(HEADS, p.G - first), h0 = hk * p.G + first;
  for (int i = threadIdx.x; i < nh * D; i += kDecWarps * 32) {
    const int hl = i / D, d = i % D;
    float M = kNoMax, MV = kNoMax;
    for (int k = from; k < last + (ended ? 1 : 0); ++k) {
      if (k != last && s_tail[k] != item) continue;  // a warp without tiles
      const float4 st = s_stat[(k * 2 + (k == last ? 0 : 1)) * HEADS + hl];
      M = fmaxf(M, st.x);
      MV = fmaxf(MV, st.y);
    }
    float L = 0.f, A = 0.f;
    for (int k = from; k < last + (ended ? 1 : 0); ++k) {
      if (k != last && s_tail[k] != item) continue;
      const float4 st = s_stat[(k * 2 + (k == last ? 0 : 1)) * HEADS + hl];
      const float* src = k == last ? warp_part + (size_t)k * p.part_stride
                                   : reinterpret_cast<const float*>(smem + k * Cfg::STAGES * Cfg::STAGE_BYTES);
      L += st.z * exp2f(st.x - M);
      A += src[i] * exp2f(st.y - MV);
    }
    if (dst == nullptr) {
      const size_t oi = (size_t)token * p.H + h0 + hl;
      p.out[oi * D + d] = __float2bfloat16(L == 0.f ? 0.f : A * final_factor(M, MV, L));
      if (d == 0 && p.lse != nullptr) p.lse[oi] = final_lse(M, L);
    } else {
      dst[i] = A;
      if (d == 0) reinterpret_cast<float4*>(dst + p.part_heads * D)[hl] = make_float4(M, MV, L, 0.f);
    }
  }
}

// ---------------------------------------------------------------------------
// Main kernel. Per tile and warp: the codes of TR rows of K and V come through
// a ring in shared memory that cp.async fills STAGES - 1 tiles ahead; every lane
// copies just the bytes that it will hold in MMA fragments, so neither a bank
// conflict nor a barrier stands between copy and use. S^T = K Q^T has the rows as
// M and the heads as N: codes convert to the fp16 A operand exactly, K's
// contraction index runs over d in whatever order the lanes hold it (Q follows).
// O^T = V^T P^T takes V's codes of two rows interleaved by byte as its A
// operand, and P through a register transpose.
//
// V's scale enters through the exponent: p' = 2^(s + log2 vscale - mv) with its
// own running maximum mv, so pages of any two sizes keep their precision, and
// the softmax sum uses p = 2^(s - m) in fp32. p' is rounded to fp16 for the
// product (2^-11 relative, below the bf16 rounding of the result).
// ---------------------------------------------------------------------------
template <int D, int NB, int FMT>
__global__ void __launch_bounds__(kDecWarps * 32, (DecodeCfg<D, NB>::BLOCKS_PER_SM))
    decode_kernel(const __grid_constant__ DecodeParams p) {
  using Cfg = DecodeCfg<D, NB>;
  constexpr int TR = Cfg::TR, RB = Cfg::RB, HEADS = Cfg::HEADS, ST = Cfg::STAGES;
  constexpr int MT = D / 16;       // M tiles of O^T; k-steps of S
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  float4* s_stat = reinterpret_cast<float4*>(smem + Cfg::RING_BYTES);  // [warp][head, tail][HEADS]
  int* s_head = reinterpret_cast<int*>(s_stat + Cfg::STATS);  // [warp] item from before that ends here
  int* s_tail = s_head + kDecWarps;                           // [warp] item that goes on past its range
  int* s_mid = s_tail + kDecWarps;                            // [warp] that item began before its range
  if (lane == 0) s_head[warp] = s_tail[warp] = -1;

  grid_dependency_wait();
  // ---- this warp's range of the tile sequence
  const int groups = (p.items + p.group - 1) / p.group;
  long long* s_sum = reinterpret_cast<long long*>(smem);  // inclusive sums over groups
  {
    long long* s_warp = s_sum + kDecGroups;
    long long v[4], run = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = tid * 4 + i;
      run += k < groups ? p.sums[k] : 0;
      v[i] = run;
    }
    long long x = run;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, s);
      if (lane >= s) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = x - run;
    for (int i = 0; i < warp; ++i) before += s_warp[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) s_sum[tid * 4 + i] = before + v[i];
    __syncthreads();
  }
  const long long total = s_sum[kDecGroups - 1];
  // at least two tiles for each warp of a block that works
  const long long want = (total + 2 * kDecWarps - 1) / (2 * kDecWarps);
  const int nblk = (int)min((long long)gridDim.x, want);
  const int bid = blockIdx.x;
  long long cta0 = 0, cta1 = 0;
  if (bid < nblk) {
    cta0 = total * bid / nblk;
    cta1 = total * (bid + 1) / nblk;
  }
  const long long t0 = cta0 + (cta1 - cta0) * warp / kDecWarps;
  const long long t1 = cta0 + (cta1 - cta0) * (warp + 1) / kDecWarps;
  int item0 = 0, tile0 = 0;
  if (t0 < t1) {
    int a = 0, e = groups - 1;  // first group whose inclusive sum is above t0
    while (a < e) {
      const int m = (a + e) >> 1;
      if (s_sum[m] > t0) e = m; else a = m + 1;
    }
    long long at = a > 0 ? s_sum[a - 1] : 0;
    int i = a * p.group;
    const int end = min(i + p.group, p.items);
    for (;; i += 32) {
      const int cnt = i + lane < end ? p.counts[i + lane] : 0;
      int x = cnt;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, s);
        if (lane >= s) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + x > t0);
      if (past != 0 || i + 32 >= end) {
        const int k = past != 0 ? __ffs(past) - 1 : 0;
        item0 = i + k;
        tile0 = (int)(t0 - at - __shfl_sync(0xffffffffu, x - cnt, k));
        break;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();  // the ring takes the sums' place
  grid_dependency_release();

  // ---- the warp's walk
  const uint32_t ring = smem_u32(smem) + warp * ST * Cfg::STAGE_BYTES;
  const uint8_t* ring_p = smem + warp * ST * Cfg::STAGE_BYTES;
  float* wpart = p.warp_part + ((size_t)bid * kDecWarps + warp) * p.part_stride;
  const int row_l = TR == 16 ? (lane & 15) : lane;  // the row this lane looks up
  DecodeItem ahead, it;      // items of the tile to fetch next and of the tile in hand
  int a_item = item0, a_tile = tile0;
  long long a_left = t1 - t0;
  int f_page = -1, f_x = 0, f_hk = 0;  // looked-up page of the tile to copy next
  bool f_some = false;
  if (a_left > 0) load_item<TR, HEADS>(p, a_item, ahead);

  // look up the pages of the next tile's rows
  auto look_up = [&]() {
    f_some = a_left > 0;
    if (!f_some) return;
    const int j = __popc(__ballot_sync(0xffffffffu, lane < p.npat && a_tile >= ahead.tend));
    const int jj = min(j, p.npat - 1);
    const int tstart = jj > 0 ? __shfl_sync(0xffffffffu, ahead.tend, jj - 1) : 0;
    const int n = j < p.npat ? __shfl_sync(0xffffffffu, ahead.n, jj) : 0;
    const int base = __shfl_sync(0xffffffffu, ahead.base, jj);
    const uint32_t k = (uint32_t)(a_tile - tstart) * TR + row_l;  // may pass 2^31 in the last tile
    f_page = -1;
    f_hk = ahead.hk;
    if (k < (uint32_t)n) {
      f_x = base + (int)k * p.r[jj];
      f_page = p.geom.table[(size_t)ahead.b * p.geom.max_pages + (f_x >> p.geom.lp)];
      if ((unsigned)f_page >= (unsigned)p.geom.pages) {
        p.geom.err.raise(kErrBadPage);
        f_page = -1;
      }
    }
    --a_left;
    if (++a_tile == ahead.tiles && a_left > 0) {
      a_tile = 0;
      load_item<TR, HEADS>(p, ++a_item, ahead);
    }
  };
  // copy the looked-up tile into ring stage st
  auto copy = [&](int st) {
    if (f_some) {
      const uint32_t blk = (uint32_t)f_page * (uint32_t)p.geom.Hkv + (uint32_t)f_hk;
      const bool in = f_page >= 0;
      const uint32_t idx = in ? (blk << p.geom.lp) + (uint32_t)(f_x & ((1 << p.geom.lp) - 1)) : 0xffffffffu;
      const uint32_t dst = ring + st * Cfg::STAGE_BYTES;
      const uint32_t sc = dst + 2 * TR * D;
      const size_t so = in ? blk : 0;
      if constexpr (TR == 16) {
        cp_async4(sc + lane * 4, p.scale[lane >> 4] + so, in);
      } else {
        cp_async4(sc + lane * 4, p.scale[0] + so, in);
        cp_async4(sc + 128 + lane * 4, p.scale[1] + so, in);
      }
#pragma unroll
      for (int i = 0; i < 2 * RB; ++i) {  // K rows g, g + 8 (, g + 16, g + 24)
        const uint32_t x = __shfl_sync(0xffffffffu, idx, i * 8 + g);
        const bool ok = x != 0xffffffffu;
        const uint8_t* src = p.codes[0] + (ok ? (size_t)x * D : 0) + c * 16;
#pragma unroll
        for (int q = 0; q < D / 64; ++q)
          cp_async16(dst + (i * (D / 64) + q) * 512 + lane * 16, src + q * 64, ok);
      }
      const uint32_t dv = dst + TR * D;
#pragma unroll
      for (int i = 0; i < 4 * RB; ++i) {  // V rows 2c, 2c + 1, 2c + 8, 2c + 9 of each 16
        const int row = (i >> 2) * 16 + ((i >> 1) & 1) * 8 + 2 * c + (i & 1);
        const uint32_t x = __shfl_sync(0xffffffffu, idx, row);
        const bool ok = x != 0xffffffffu;
        const uint8_t* src = p.codes[1] + (ok ? (size_t)x * D : 0) + g * (D / 8);
        if constexpr (D == 128) cp_async16(dv + i * 512 + lane * 16, src, ok);
        else cp_async8(dv + i * 256 + lane * 8, src, ok);
      }
    }
    cp_async_commit();
  };

  float acc[MT][NB][4];
  float m[2 * NB], mv[2 * NB], l[2 * NB], fac[2 * NB];
  uint32_t qf[NB][MT][2];
  uint32_t in_pat[2 * NB];  // patterns that each of the lane's heads takes part in
  // heads of this lane: nb * 8 + 2 c + e
  auto begin_item = [&](int item) {
    load_item<TR, HEADS>(p, item, it);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      // q of head nb * 8 + g, lifted by a power of two to [2^13, 2^14): exact in fp16
      // (elements under 2^-37 of the largest are cut)
      const int hl = nb * 8 + g;
      uint2 raw[MT];
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int d0 = (k >> 2) * 64 + c * 16 + (k & 3) * 4;
        raw[k] = hl < it.nh ? *reinterpret_cast<const uint2*>(p.q + (long long)it.token * p.q_stride +
                                                              (it.h0 + hl) * D + d0)
                            : make_uint2(0, 0);
        big = max(max(big, raw[k].x & 0x7fffu), (raw[k].x >> 16) & 0x7fffu);
        big = max(max(big, raw[k].y & 0x7fffu), (raw[k].y >> 16) & 0x7fffu);
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // exponent of the largest; subnormal and zero count as the smallest normal one
      const int e = max((int)(big >> 7), 1) - 127;
      // 2^(13 - e) in two factors that fp32 holds
      const int up = 13 - e, u1 = up / 2, u2 = up - u1;
      const float f1 = __uint_as_float((uint32_t)(u1 + 127) << 23), f2 = __uint_as_float((uint32_t)(u2 + 127) << 23);
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const __half2 a = __floats2half2_rn(__uint_as_float(raw[k].x << 16) * f1 * f2,
                                            __uint_as_float(raw[k].x & 0xffff0000u) * f1 * f2);
        const __half2 b = __floats2half2_rn(__uint_as_float(raw[k].y << 16) * f1 * f2,
                                            __uint_as_float(raw[k].y & 0xffff0000u) * f1 * f2);
        qf[nb][k][0] = *reinterpret_cast<const uint32_t*>(&a);
        qf[nb][k][1] = *reinterpret_cast<const uint32_t*>(&b);
      }
      const float down = big >= 0x7f80u ? __uint_as_float(0x7fffffffu)  // NaN or infinity in q
                                        : p.qk_scale / f1 / f2;
      fac[2 * nb] = __shfl_sync(0xffffffffu, down, 8 * c);
      fac[2 * nb + 1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2) {
        m[2 * nb + e2] = mv[2 * nb + e2] = kNoMax;
        l[2 * nb + e2] = 0.f;
        in_pat[2 * nb + e2] = 0;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = __ballot_sync(0xffffffffu, it.heads >> (nb * 8 + k) & 1u);
        if ((k >> 1) == c) in_pat[2 * nb + (k & 1)] = b;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[mt][nb][k] = 0.f;
    }
  };

  // where a lane's sums of one of its heads lie: d = g (D / 8) + 0 .. D / 8 - 1
  auto sum_of = [&](int nb, int e, int k) { return acc[k >> 1][nb][(k & 1) * 2 + e]; };

  // the item is done here or goes on elsewhere; `whole`: this warp had all of it
  auto end_item = [&](int item, bool whole, bool ends) {
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
    }
    if (whole) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * nb + e, hl = nb * 8 + 2 * c + e;
          if (hl >= it.nh) continue;
          const float f = final_factor(m[i], mv[i], l[i]);
          const size_t oi = (size_t)it.token * p.H + it.h0 + hl;
          uint32_t o[D / 16];
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            // no row: 0, whatever the sums hold
            const __nv_bfloat162 v = l[i] == 0.f ? __floats2bfloat162_rn(0.f, 0.f)
                : __floats2bfloat162_rn(sum_of(nb, e, 2 * k) * f, sum_of(nb, e, 2 * k + 1) * f);
            o[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.out + oi * D + g * (D / 8));
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (g == 0 && p.lse != nullptr) p.lse[oi] = final_lse(m[i], l[i]);
        }
      return;
    }
    // a tail stays in the warp's part of the ring, a head goes to the workspace
    if (!ends) {
      cp_async_wait<0>();
      __syncwarp();
    }
    float* dst = ends ? wpart : reinterpret_cast<float*>(smem + warp * ST * Cfg::STAGE_BYTES);
    float4* stat = s_stat + (warp * 2 + (ends ? 0 : 1)) * HEADS;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * nb + e, hl = nb * 8 + 2 * c + e;
        if (hl >= it.nh) continue;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          *reinterpret_cast<float4*>(dst + hl * D + g * (D / 8) + 4 * k) =
              make_float4(sum_of(nb, e, 4 * k), sum_of(nb, e, 4 * k + 1), sum_of(nb, e, 4 * k + 2),
                          sum_of(nb, e, 4 * k + 3));
        if (g == 0) stat[hl] = make_float4(m[i], mv[i], l[i], 0.f);
      }
    if (lane == 0) (ends ? s_head : s_tail)[warp] = item;
  };

  if (t0 < t1) {
    look_up();
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      copy(s);
      look_up();
    }
    int item = item0, tile = tile0, st = 0;
    bool from_start = tile0 == 0;
    begin_item(item);
    for (long long left = t1 - t0; left > 0; --left) {
      cp_async_wait<ST - 2>();
      __syncwarp();
      {
        int nx = st + ST - 1;
        if (nx >= ST) nx -= ST;
        copy(nx);
        look_up();
      }
      const uint8_t* kp = ring_p + st * Cfg::STAGE_BYTES;
      const uint8_t* vp = kp + TR * D;
      const float* sp = reinterpret_cast<const float*>(vp + TR * D);

      // ---- which rows count, and how often
      const int j = __popc(__ballot_sync(0xffffffffu, lane < p.npat && tile >= it.tend));
      uint32_t held = 1;  // patterns that hold this lane's row
      if (p.npat > 1) {
        const int jj = min(j, p.npat - 1);
        const int tstart = jj > 0 ? __shfl_sync(0xffffffffu, it.tend, jj - 1) : 0;
        // rows past the walk's end wrap or lie past the token: they have no scale
        const int x = (int)((uint32_t)__shfl_sync(0xffffffffu, it.base, jj) +
                            (uint32_t)((tile - tstart) * TR + row_l) * (uint32_t)p.r[jj]);
        const int dist = (int)((uint32_t)it.pos - (uint32_t)x);
        held = 0;
        for (int i = 0; i < p.npat; ++i) {
          const int si = __shfl_sync(0xffffffffu, it.s, i);
          if (x >= si && divides(p, i, dist)) held |= 1u << i;
        }
      }
      const uint32_t upto = (2u << j) - 1, mine = 1u << j;

#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        // ---- scores: rows rb * 16 + g and + 8, heads nb * 8 + 2 c and + 1
        float sc[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[nb][k] = 0.f;
#pragma unroll
        for (int q = 0; q < D / 64; ++q) {
          const uint4 ka = *reinterpret_cast<const uint4*>(kp + ((2 * rb) * (D / 64) + q) * 512 + lane * 16);
          const uint4 kb = *reinterpret_cast<const uint4*>(kp + ((2 * rb + 1) * (D / 64) + q) * 512 + lane * 16);
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a0, a1, a2, a3;
            codes_to_half<FMT>(wa[k], a0, a2);
            codes_to_half<FMT>(wb[k], a1, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_16816(sc[nb], a0, a1, a2, a3, qf[nb][q * 4 + k][0], qf[nb][q * 4 + k][1]);
          }
        }
        // ---- softmax weights
        float cnt[NB][4], sv[NB][4];
        bool raise = false;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {  // row half
          const int row = rb * 16 + hf * 8 + g;
          const float ks = sp[row];
          const float lv = fast_log2(sp[TR + row]);
          const uint32_t hr = __shfl_sync(0xffffffffu, held, row);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = hf * 2 + e, i = 2 * nb + e;
              const uint32_t u = hr & in_pat[i];
              // rows that are not there were filled with zeros: no scale is zero
              const bool ok = (u & upto) == mine && ks != 0.f;
              cnt[nb][k] = (float)__popc(u);
              const float s = ok ? sc[nb][k] * (fac[i] * ks) : -INFINITY;
              sc[nb][k] = s;
              sv[nb][k] = ok ? s + lv : -INFINITY;
              raise = raise || s > m[i] + kMaxSlack || sv[nb][k] > mv[i] + kMaxSlack;
            }
        }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = 2 * nb + e;
              float a = fmaxf(sc[nb][e], sc[nb][2 + e]), b = fmaxf(sv[nb][e], sv[nb][2 + e]);
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, s));
                b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, s));
              }
              a = fmaxf(a, m[i]);
              b = fmaxf(b, mv[i]);
              l[i] *= fast_exp2(m[i] - a);
              const float f = fast_exp2(mv[i] - b);
              m[i] = a;
              mv[i] = b;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                acc[mt][nb][e] *= f;
                acc[mt][nb][2 + e] *= f;
              }
            }
        }
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float pv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = hf * 2 + e, i = 2 * nb + e;
              l[i] += fast_exp2(sc[nb][k] - m[i]) * cnt[nb][k];
              pv[e] = fast_exp2(sv[nb][k] - (mv[i] - kPBias)) * cnt[nb][k];
            }
            const __half2 h2 = __floats2half2_rn(pv[0], pv[1]);
            pf[nb][hf] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h2));
          }
        // ---- O^T += V^T P^T
        constexpr int VW = D / 32;  // 32-bit words of a row that a lane holds
        uint32_t vr[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(vp + (rb * 4 + i) * 512 + lane * 16);
            vr[i][0] = u.x, vr[i][1] = u.y, vr[i][2] = u.z, vr[i][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(vp + (rb * 4 + i) * 256 + lane * 8);
            vr[i][0] = u.x, vr[i][1] = u.y;
          }
        }
#pragma unroll
        for (int k = 0; k < VW; ++k)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            codes_to_half<FMT>(__byte_perm(vr[0][k], vr[1][k], sel), a0, a1);
            codes_to_half<FMT>(__byte_perm(vr[2][k], vr[3][k], sel), a2, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_16816(acc[2 * k + half][nb], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
          }
      }
      if (++st == ST) st = 0;
      const bool ends = ++tile == it.tiles;
      if (ends || left == 1) {
        if (lane == 0) s_mid[warp] = !from_start;
        end_item(item, ends && from_start, ends);
        if (left > 1) {
          tile = 0;
          from_start = true;
          begin_item(++item);
        }
      }
    }
  }

  // ---- join the block's warps. A run is an item's partials of successive
  // warps: tails, and the head that ends it unless it goes on in the next block.
  __syncthreads();
  int run = -1, from = 0, begun = -1, unfinished = -1;
  bool before = false;  // the run's item began before the block's range
  for (int w = 0; w <= kDecWarps; ++w) {
    const int head = w < kDecWarps ? s_head[w] : -1;
    const bool ended = head >= 0;
    if (ended && run < 0) {
      run = head;
      from = w;
      before = true;
    }
    if (run >= 0 && (ended || w == kDecWarps)) {
      float* dst = nullptr;
      if (!ended || before) {
        dst = p.part + ((size_t)bid * 2 + (before ? 0 : 1)) * p.part_stride;
        if (before) begun = run; else unfinished = run;
      }
      join_warps<D, NB>(p, run, from, w, ended, s_tail, s_stat, smem,
                        p.warp_part + (size_t)bid * kDecWarps * p.part_stride, dst);
      run = -1;
    }
    if (w < kDecWarps && s_tail[w] >= 0 && run < 0) {
      run = s_tail[w];
      from = w;
      before = s_mid[w] != 0;
    }
  }
  if (tid == 0) {
    p.begun[bid] = begun;
    p.unfinished[bid] = unfinished;
  }
}

// ---------------------------------------------------------------------------
// Join of items cut between blocks: block (b, head) takes the item that begins
// in block b of the main kernel and ends past it, with the partials of the
// blocks behind it in order.
// ---------------------------------------------------------------------------
template <int D, int NB>
__global__ void __launch_bounds__(D) decode_join_kernel(const __grid_constant__ DecodeParams p,
                                                        int blocks) {
  using Cfg = DecodeCfg<D, NB>;
  constexpr int HEADS = Cfg::HEADS;
  __shared__ int s_n;
  grid_dependency_wait();
  const int b0 = blockIdx.x, hl = blockIdx.y, tid = threadIdx.x;
  const int item = p.unfinished[b0];
  if (item < 0) return;
  const int token = item / p.per_token, cc = item % p.per_token;
  const int hk = cc / p.nsub, sub = cc % p.nsub;
  if (hl >= min(HEADS, p.G - sub * HEADS)) return;
  if (tid == 0) s_n = blocks - b0 - 1;
  __syncthreads();
  for (int i = tid; b0 + 1 + i < blocks; i += D)
    if (p.begun[b0 + 1 + i] != item) {
      atomicMin(&s_n, i);
      break;
    }
  __syncthreads();
  const int n = s_n;  // further blocks
  const float* first = p.part + ((size_t)b0 * 2 + 1) * p.part_stride;
  const float* rest = p.part + (size_t)(b0 + 1) * 2 * p.part_stride;
  const size_t step = (size_t)2 * p.part_stride;
  const int so = p.part_heads * D + hl * 4;
  const float4 f = *reinterpret_cast<const float4*>(first + so);
  float M = f.x, MV = f.y;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float2 st = *reinterpret_cast<const float2*>(rest + i * step + so);
    M = fmaxf(M, st.x);
    MV = fmaxf(MV, st.y);
  }
  float L = f.z * exp2f(f.x - M);
  float A = first[hl * D + tid] * exp2f(f.y - MV);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 st = *reinterpret_cast<const float4*>(rest + i * step + so);
    L += st.z * exp2f(st.x - M);
    A += rest[i * step + hl * D + tid] * exp2f(st.y - MV);
  }
  const size_t oi = (size_t)token * p.H + hk * p.G + sub * HEADS + hl;
  p.out[oi * D + tid] = __float2bfloat16(L == 0.f ? 0.f : A * final_factor(M, MV, L));
  if (tid == 0 && p.lse != nullptr) p.lse[oi] = final_lse(M, L);
}

}  // namespace dil
