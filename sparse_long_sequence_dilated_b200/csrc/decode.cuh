// Dilated attention of single query tokens over the 8-bit paged cache.
//
// Which rows. A token at position t takes part in pattern (w, r) for the heads
// h with h mod r = (t - s) mod r, s = floor(t / w) w its segment's start; those
// heads then all attend the same rows: t, t - r, t - 2 r, ... down to s. The
// output is one softmax over the multiset union of the patterns' rows, so a row
// that several patterns hold is read once and weighted by their number.
//
// Items. An item is a (token, KV head) pair with up to 16 of the query heads
// that share the KV head: they share its rows too.
// Patterns are sorted by r. A row is walked by the first pattern, for that
// head, that holds it. Where r_l divides r_j and every head of the item that
// takes part in j takes part in l, l walks all of j's rows from s_l on, so j's
// walk ends there; what overlap remains (r that do not divide one another) is
// masked row by row. An item's walks, in tiles of 32 rows, are its work.
//
// Dense attention of several tokens to a sequence (drafted tokens) reads the
// same rows for all of them. There an item has p.tokens successive tokens, whose
// heads side by side are its columns, and a walk for each sequence among them;
// a row counts for the columns of its sequence whose token is not before it.
//
// Split. The tiles of all items form one sequence that is cut into contiguous
// ranges of equal weight, one for each warp of a persistent grid, wherever the cut
// falls: no batch shape, length or head count leaves SMs idle. Warps do not
// wait for one another. An item inside one range is finished by its warp; an
// item that is cut leaves partials that a join kernel combines in warp
// order (no atomics: the same call gives the same bits).
//
// What bounds it. Every distinct row is 2 d bytes for 4 d operations a head, far
// below the machine's balance: the cache's bytes at the copy rate are the floor,
// and bytes under way what a warp has to keep up. mma.sync serves that: its
// 16-row tiles fit any row list and any number of heads from one on, the tensor
// pipe is 11 to 18% busy, and nothing has to pass through shared memory or TMEM.
// 1,048,576 tokens of 8 KV heads with 4 query heads each, d = 128 (2.1 GB), take
// 390 us as a call among others (5.5 TB/s), and 340 to 350 replayed from a graph
// (6.1 TB/s), where a ring of tiles in shared memory filled by cp.async (three
// stages, 16 warps) took 440.
//
// Launches: few or short items have decode_team_kernel alone. Otherwise
// decode_plan_kernel, one block or cluster, describes every item's walks once
// and cuts the sequence (above kPlanBlocks * kPlanThreads items,
// decode_walks_kernel describes them before it, over the whole GPU), then
// decode_kernel, then a join kernel. Each is launched while the one before
// it runs and waits for that one's end.
#pragma once

#include <cooperative_groups.h>

#include "cache.cuh"

namespace dil {

constexpr int kDecWarps = 4;         // warps of a block
constexpr int kDecMaxSms = 160;      // the workspace has partials for the warps of this many SMs
constexpr int kDecTile = 32;         // rows of a tile
constexpr int kPlanBlocks = 8;       // blocks of the plan's cluster
constexpr int kPlanThreads = 512;    // threads of one of them, and the most groups of items that it has
constexpr int kPlanAlone = 1024;     // threads of a plan of one block
constexpr int kWalkThreads = 256;

// What a warp's time goes by, in quarters of a tile whose rows lie side by side:
// a tile of spread rows (r > 1) takes 1.26 to 1.36 times as long at d = 64 and
// 1.21 to 1.39 times at d = 128, the beginning of an item 0.7 and 0.5 of a tile (a
// least-squares fit over the warps of ragged batches with 5 and 7 patterns).
constexpr int kTileWeight = 4, kSpreadWeight = 5, kItemWeight = 2;
// Two cuts so far apart have the beginning of a tile between them.
constexpr int kRangeWeight = 8;

// Where a warp's range of the tile sequence begins: at tile `tile` of item `item`.
// The range ends where the next one begins.
struct __align__(8) DecodeRange {
  int item, tile;
};
// One walk of an item: rows base + k r, k < n. s: the segment's start (the
// largest int when no head of the item takes part; with p.tokens > 1 the
// sequence); heads: bits of those that take part.
struct __align__(16) DecodeWalk {
  int s, n, base;
  uint32_t heads;
};
struct __align__(16) DecodeHead {
  int b, pos, tiles, pad;
};

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
  int heads;                 // most columns of an item: 1, 2, 4, 8 or 16
  int nsub;                  // items that a KV head's query heads make up
  int per_token;             // Hkv * nsub
  uint32_t pt_mul, ns_mul;   // reciprocals of per_token and nsub (divisor_magic)
  int pt_sh, ns_sh;
  int items;
  int group;                 // items of a group: 1, or what a block of decode_walks_kernel describes
                             // (a multiple of kWalkThreads / lanes)
  int lanes;                 // threads that describe an item: a power of two, at least npat
  int warps;                 // warps of the grid
  int team;                  // blocks that share an item in decode_team_kernel; 0: a warp for each item
  float qk_scale;            // log2(e) / sqrt(d)
  int npat;                  // patterns, by ascending r
  int dense;                 // one pattern with r = 1: every head of a token takes every row of a walk
  int tokens;                // tokens of an item
  int g_rec;                 // ceil(256 / G): i / G = i g_rec / 256 for i < 16, G <= 8
  int w[kMaxPat], r[kMaxPat];
  uint32_t w_mul[kMaxPat], r_mul[kMaxPat];
  int w_sh[kMaxPat], r_sh[kMaxPat];
  uint32_t r_inv[kMaxPat], r_lim[kMaxPat];  // divisibility by r (see divides)
  int r_rot[kMaxPat];
  uint32_t divisors[kMaxPat];               // earlier patterns whose r divides this one's
  // workspace
  DecodeHead* head;          // [items]
  DecodeWalk* walk;          // [items][npat]
  long long* upto;           // [items] weight of the item's group up to and including it
  long long* sums;           // [groups] weight of each group
  DecodeRange* range;        // [warps + 1]
  float* part;               // [warps][2]: an item that began before the range; one that goes on past it
  int part_heads, part_stride;  // heads and floats of a partial: sums [heads][D], (m, mv, l, -) [heads]
};

// x mod r == 0, for x < 2^31 and r = 2^rot odd: x times the inverse of odd
// modulo 2^32, rotated right by rot, is x / r when r divides x and more than
// (2^32 - 1) / r otherwise (Granlund and Montgomery 1994, section 9).
__device__ __forceinline__ bool divides(const DecodeParams& p, int i, int x) {
  const uint32_t y = (uint32_t)x * p.r_inv[i];
  return __funnelshift_r(y, y, p.r_rot[i]) <= p.r_lim[i];
}

// Blocks of the main kernel on an SM, by registers: 128, 168 or 255 a thread. What
// does not fit is loads under way, and a spill of one waits for it: eight columns
// of drafts at d = 128 take 130 us with two blocks and 212 us with three.
constexpr int decode_blocks_per_sm(int d, int heads, bool grouped) {
  return heads > 8 || (d == 128 && grouped) ? 2 : d == 64 ? 4 : 3;
}

// What a kernel is made for: any patterns (dense ones too), one dense pattern and
// a token to an item (which spares the counting of patterns for every score), and
// one dense pattern and several tokens to an item.
enum DecodeMode : int { kAnyPatterns = 0, kDense = 1, kGrouped = 2 };

// Where an item belongs; nh: its columns. `tokens` is p.tokens, or 1 where that is known.
struct DecodeItem {
  int token, hk, h0, nh;
};
__device__ __forceinline__ DecodeItem item_of(const DecodeParams& p, int item, int tokens) {
  DecodeItem it;
  it.token = (int)udiv((uint32_t)item, p.pt_mul, p.pt_sh);
  const int c = item - it.token * p.per_token;
  it.hk = (int)udiv((uint32_t)c, p.ns_mul, p.ns_sh);
  const int first = (c - it.hk * p.nsub) * p.heads;
  it.h0 = it.hk * p.G + first;
  it.nh = min(p.heads, p.G - first);
  if (tokens > 1) {
    it.token *= tokens;
    it.nh = min(tokens, p.T - it.token) * p.G;
  }
  return it;
}
// The token of an item's column, and where in [T][H] its head lies.
__device__ __forceinline__ int token_of(const DecodeParams& p, const DecodeItem& it, int column, int tokens) {
  return it.token + (tokens > 1 ? column * p.g_rec >> 8 : 0);
}
__device__ __forceinline__ int head_of(const DecodeParams& p, const DecodeItem& it, int column, int tokens) {
  return it.h0 + column - (tokens > 1 ? (column * p.g_rec >> 8) * p.G : 0);
}
__device__ __forceinline__ size_t place_of(const DecodeParams& p, const DecodeItem& it, int column, int tokens) {
  return (size_t)token_of(p, it, column, tokens) * p.H + head_of(p, it, column, tokens);
}

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------
// Codes: read once by one lane each, so L1 keeps none of them.
__device__ __forceinline__ uint4 load_codes16(const uint8_t* src) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(src));
  return x;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* src) {
  uint2 x;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(src));
  return x;
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

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------

// Writes an item's head and walks; returns its weight. p.lanes threads
// of a warp work on an item, lane j of them on pattern j; all 32 take part.
__device__ int describe_item(const DecodeParams& p, int item, DecodeHead* head, DecodeWalk* walk) {
  const bool real = item < p.items;
  const DecodeItem it = item_of(p, real ? item : 0, p.tokens);
  const int j = threadIdx.x & (p.lanes - 1), jj = min(j, p.npat - 1);
  const int token = it.token + (p.tokens > 1 ? j : 0);
  DecodeHead hd;
  hd.b = 0;
  hd.pos = -1;
  if (token < p.T && (p.tokens == 1 || j < p.tokens)) {  // lanes may be more than the tokens
    hd.b = p.seq != nullptr ? p.seq[token] : token;
    hd.pos = p.pos[token];
  }
  hd.pad = 0;
  const int r = p.r[jj], w = p.w[jj], r_sh = p.r_sh[jj];
  const uint32_t r_mul = p.r_mul[jj], w_mul = p.w_mul[jj], div = p.divisors[jj];
  const int w_sh = p.w_sh[jj];
  const int skip = it.h0 - (int)udiv((uint32_t)it.h0, r_mul, r_sh) * r;  // h0 mod r
  if (hd.pos >= 0 &&
      ((unsigned)hd.b >= (unsigned)p.geom.B || (hd.pos >> p.geom.lp) >= p.geom.max_pages)) {
    if (real) p.geom.err.raise(kErrBadPage);
    hd.pos = -1;
  }
  if (hd.pos < 0) hd.b = 0;
  DecodeWalk wk{0x7fffffff, 0, 0, 0u};
  if (p.tokens > 1) {  // the first token of a sequence walks for all
    bool first = hd.pos >= 0;
    int top = -1;
    for (int l = 0; l < p.lanes; ++l) {
      const int bl = __shfl_sync(0xffffffffu, hd.b, l, p.lanes), pl = __shfl_sync(0xffffffffu, hd.pos, l, p.lanes);
      if (bl != hd.b || pl < 0) continue;
      first = first && l >= j;
      top = max(top, pl);
      wk.heads |= ((1u << p.G) - 1) << (l * p.G);
    }
    if (first) {
      wk.s = hd.b;
      wk.n = top + 1;
    } else {
      wk.heads = 0;
    }
  }
  int s = 0;
  if (p.tokens == 1 && hd.pos >= 0 && j < p.npat) {
    s = (int)udiv((uint32_t)hd.pos, w_mul, w_sh) * w;
    const int rel = hd.pos - s;
    const int steps = (int)udiv((uint32_t)rel, r_mul, r_sh);
    const int off = rel - steps * r;
    if (r == 1) {
      wk.heads = (1u << it.nh) - 1;
    } else {
      for (uint32_t k = off < skip ? off - skip + r : off - skip; k < (uint32_t)it.nh; k += (uint32_t)r)
        wk.heads |= 1u << k;  // k + r stays below 2^32
    }
    if (wk.heads != 0) {
      wk.s = s;
      wk.base = s + off;
      wk.n = steps + 1;
    }
  }
  int limit = 0x7fffffff;
  for (int l = 0; l + 1 < p.npat && p.tokens == 1; ++l) {
    const int sl = __shfl_sync(0xffffffffu, s, l, p.lanes);
    const uint32_t hl = __shfl_sync(0xffffffffu, wk.heads, l, p.lanes);
    if ((div >> l & 1u) && (wk.heads & ~hl) == 0) limit = min(limit, sl);
  }
  if (p.tokens == 1 && wk.n > 0 && limit <= hd.pos)
    wk.n = limit > wk.base ? (int)udiv((uint32_t)(limit - 1 - wk.base), r_mul, r_sh) + 1 : 0;
  if (real && j < p.npat) walk[j] = wk;
  int tiles = (int)(((uint32_t)wk.n + kDecTile - 1) / kDecTile);
  int weight = tiles * (r == 1 ? kTileWeight : kSpreadWeight);
  for (int d = 1; d < p.lanes; d <<= 1) {
    tiles += __shfl_xor_sync(0xffffffffu, tiles, d);
    weight += __shfl_xor_sync(0xffffffffu, weight, d);
  }
  // an item without rows keeps one empty tile: the warp that has it writes its zeros
  hd.tiles = max(tiles, 1);
  if (real && j == 0) *head = hd;
  return kItemWeight + max(weight, kTileWeight);
}

// The first tile of an item that begins at or after this weight of it.
__device__ __forceinline__ DecodeRange tile_at(const DecodeParams& p, int item, int at) {
  const int tiles = p.head[item].tiles;
  at -= kItemWeight;
  if (at <= 0) return DecodeRange{item, 0};
  int tile = 0;
#pragma unroll 4
  for (int j = 0; j < p.npat; ++j) {
    const int n = (int)(((uint32_t)p.walk[(size_t)item * p.npat + j].n + kDecTile - 1) / kDecTile);
    const int before = p.r[j] == 1 ? (at + kTileWeight - 1) / kTileWeight : (at + kSpreadWeight - 1) / kSpreadWeight;
    tile += at > 0 ? min(before, n) : 0;
    at -= n * (p.r[j] == 1 ? kTileWeight : kSpreadWeight);
  }
  // past the last one's beginning: the next item's first
  return at > 0 || tile >= tiles ? DecodeRange{item + 1, 0} : DecodeRange{item, tile};
}

// Inclusive sums over a block's threads; s_warp: one slot for each warp.
__device__ __forceinline__ long long block_scan(long long x, long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, s);
    if (lane >= s) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  long long before = lane < warp ? s_warp[lane] : 0;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) before += __shfl_xor_sync(0xffffffffu, before, s);
  return x + before;
}

// A block for each group of items, which is whole rounds of what it describes at a time.
__global__ void __launch_bounds__(kWalkThreads)
    decode_walks_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ long long s_warp[kWalkThreads / 32];
  __shared__ int s_weight[kWalkThreads];
  __shared__ long long s_run;
  grid_dependency_wait();
  grid_dependency_release();
  const int per = kWalkThreads / p.lanes, mine = threadIdx.x / p.lanes;  // items at a time
  const long long first = (long long)blockIdx.x * p.group;
  const int end = (int)min(first + p.group, (long long)p.items);
  long long run = 0;
  for (int i = (int)first; i < end; i += per) {
    const int item_l = i + mine;
    const int weight = describe_item(p, item_l, p.head + item_l, p.walk + (size_t)item_l * p.npat);
    if ((threadIdx.x & (p.lanes - 1)) == 0) s_weight[mine] = weight;
    __syncthreads();
    const int item = i + threadIdx.x;
    const bool real = threadIdx.x < per && item < end;
    const long long x = run + block_scan(real ? s_weight[threadIdx.x] : 0, s_warp);
    if (real) p.upto[item] = x;
    if (threadIdx.x == kWalkThreads - 1) s_run = x;
    __syncthreads();
    run = s_run;
  }
  if (threadIdx.x == 0) p.sums[blockIdx.x] = run;
}

// a / b for numbers from 0 on, in 32 bits where they fit: a 64-bit division takes several times as long.
__device__ __forceinline__ long long divide(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// One cluster of `BLOCKS`; each block has a stretch of the groups. With p.group = 1
// the blocks describe the items themselves.
template <int BLOCKS>
__global__ void __launch_bounds__(BLOCKS > 1 ? kPlanThreads : kPlanAlone)
    decode_plan_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int THREADS = BLOCKS > 1 ? kPlanThreads : kPlanAlone;
  __shared__ long long s_sum[THREADS];  // inclusive sums over the block's groups
  __shared__ int s_weight[THREADS];
  __shared__ long long s_warp[THREADS / 32];
  __shared__ long long s_block[BLOCKS];  // every block's sum
  // the other blocks' shared memory is there once this has been waited for
  if constexpr (BLOCKS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependency_release();
  const int tid = threadIdx.x, rank = (int)blockIdx.x;
  const int groups = (int)(((long long)p.items + p.group - 1) / p.group);
  const int per = (groups + BLOCKS - 1) / BLOCKS;
  const int g0 = rank * per, g1 = min(g0 + per, groups), cnt = max(g1 - g0, 0);
  long long x = 0;
  if (p.group == 1) {
    const int at_once = THREADS / p.lanes, mine = tid / p.lanes;
    for (int i = 0; i < cnt; i += at_once) {
      if (i + (tid & ~31) / p.lanes >= cnt) break;  // a whole warp without items
      const bool real = i + mine < cnt;
      const int item = real ? g0 + i + mine : p.items;
      const int weight = describe_item(p, item, p.head + item, p.walk + (size_t)item * p.npat);
      if (real && (tid & (p.lanes - 1)) == 0) s_weight[i + mine] = weight;
    }
    __syncthreads();
    if (tid < cnt) x = s_weight[tid];
  } else if (tid < cnt) {
    x = p.sums[g0 + tid];
  }
  x = block_scan(x, s_warp);
  s_sum[tid] = x;
  long long total = 0, begin = 0;
  if constexpr (BLOCKS > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    __syncthreads();
    if (tid < BLOCKS) {
      cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
      *cluster.map_shared_rank(&s_block[rank], tid) = s_sum[THREADS - 1];
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
#pragma unroll
    for (int k = 0; k < BLOCKS; ++k) {
      if (k == rank) begin = total;
      total += s_block[k];
    }
  } else {
    __syncthreads();
    total = s_sum[THREADS - 1];
  }
  const int n = (int)max(min((long long)p.warps, total / kRangeWeight), 1ll);
  const long long each = divide(total, n), more = total - each * n;
  if (rank == 0)  // ends of the last range, and empty ones
    for (int k = n + tid; k <= p.warps; k += THREADS) p.range[k] = DecodeRange{p.items, 0};
  // range k begins at each k + min(k, more); the first that does so at or after x
  auto first_from = [&](long long x) {
    const long long wide = more * (each + 1);
    return (int)(x <= wide ? divide(x + each, each + 1) : more + divide(x - wide + each - 1, each));
  };
  const int k1 = BLOCKS > 1 ? min(first_from(begin + s_sum[THREADS - 1]), n) : n;
  for (int k = (BLOCKS > 1 ? first_from(begin) : 0) + tid; k < k1; k += THREADS) {
    const long long t0 = each * k + min((long long)k, more);
    int a = 0, e = cnt - 1;  // first group whose inclusive sum is above t0
    while (a < e) {
      const int m = (a + e) >> 1;
      if (begin + s_sum[m] > t0) e = m; else a = m + 1;
    }
    long long at = begin + (a > 0 ? s_sum[a - 1] : 0);
    int item = g0 + a;
    if (p.group > 1) {  // and in it the first such item
      const int first = item * p.group;
      int lo = first, hi = (int)min((long long)first + p.group, (long long)p.items) - 1;
      while (lo < hi) {
        const int m = (int)(((long long)lo + hi) >> 1);
        if (at + p.upto[m] > t0) hi = m; else lo = m + 1;
      }
      if (lo > first) at += p.upto[lo - 1];
      item = lo;
    }
    p.range[k] = tile_at(p, item, (int)(t0 - at));
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
// to 2^15, within fp16. The largest one is then 2^7 or more, fp16's normal numbers
// begin at 2^-14, 2^-21 of it, and its step below them is 2^-24, 2^-31 of it.
constexpr float kMaxSlack = 4.f;
constexpr float kPBias = 7.f;

// Factor of the sums of an item's head, and its log-sum-exp.
__device__ __forceinline__ float final_factor(float m, float mv, float l) {
  return l == 0.f ? 0.f : exp2f(mv - m - kPBias) / l;
}
__device__ __forceinline__ float final_lse(float m, float l) {
  return l == 0.f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
}

// ---------------------------------------------------------------------------
// Main kernel. A warp holds the codes of one tile, 32 rows of K and V, in
// registers: every lane loads just the bytes that it needs in MMA fragments,
// the next tile's K once this tile's scores are done and its V once the sums are,
// so that a load has most of a tile's time to arrive and codes pass neither
// shared memory nor a barrier. S^T = K Q^T has the rows as M and the heads as N:
// codes convert to the fp16 A operand exactly, K's contraction index runs over d
// in whatever order the lanes hold it (Q follows). O^T = V^T P^T takes V's codes
// of two rows interleaved by byte as its A operand, and P through a register
// transpose.
//
// Lane 4 g + c looks up row 8 c + g of the tile: the row of slot c (16-row block
// c / 2, half c mod 2 of an MMA tile) in the fragments' row group g. HW heads
// fill an MMA's 8 columns: with fewer than 8, Q is repeated, every lane gets the
// scores of more than one column's worth of equal values, and each takes only
// its share of the rows for the softmax (HW = 1, 2: its own row, 4: two rows, 8:
// four), so that the softmax costs HW values a lane and not 8.
//
// V's scale enters through the exponent: p' = 2^(s + log2 vscale - mv) with its
// own running maximum mv, so no page's size can overflow, and the softmax sum
// uses p = 2^(s - m) in fp32. p' is rounded to fp16 for the product: 2^-11
// relative, below the bf16 rounding of the result, for rows down to 2^-21 of the
// largest p', and below that 2^-32 of the largest (see kPBias): what a row adds
// to a channel is lost where its p' is under that, however small the larger
// rows are in that channel.
// ---------------------------------------------------------------------------

// One warp's tiles from rg up to end. Items' heads and walks are at head[0] and
// walk[0] from item first_item on; part: the warp's two slots for partials, slot_stride
// floats apart; qf, s_walk: shared memory of the warp (the lane's own fragments
// of Q, NB * MT of them 32 apart, and the walks of the item to fetch from).
template <int D, int HEADS, int FMT, int MODE>
__device__ __forceinline__ void decode_range(const DecodeParams& p, const DecodeRange rg, const DecodeRange end,
                                             const DecodeHead* head, const DecodeWalk* walk, int first_item,
                                             float* part, size_t slot_stride, uint2* qf, DecodeWalk* s_walk) {
  constexpr int NB = (HEADS + 7) / 8;
  constexpr int MT = D / 16;                       // M tiles of O^T; k-steps of S
  constexpr int HW = HEADS < 8 ? HEADS : 8;        // heads of an MMA's columns
  constexpr int VR = HW <= 2 ? 1 : HW / 2;         // rows of a tile that a lane's softmax has
  constexpr int VE = HW == 1 ? 1 : 2;              // heads of them, for each NB
  constexpr bool GROUPED = MODE == kGrouped;
  const int tokens_of_item = GROUPED ? p.tokens : 1;
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int row_l = 8 * c + g;                     // the row this lane looks up
  const int first_slot = VR == 1 ? c : VR == 2 ? (c & 2) : 0;
  const int pmask = (1 << p.geom.lp) - 1;

  // ---- the walk to fetch from (a_...), the looked-up tile (f_...), the tile in registers
  int a_item = rg.item, a_tiles, a_pos, a_hk, a_b, a_j, a_n, a_base, a_r;  // a_tiles: of the item, in the range
  uint32_t a_k, a_walks, a_in;  // patterns with rows to walk; patterns of the item's head (HEADS = 1)
  int f_page = -1, f_x = 0, f_hk = 0, f_j = 0;
  uint32_t f_meta = 0;
  bool a_some = true, f_some = false, f_whole = false;

  auto set_walk = [&](int j) {
    const DecodeWalk wk = s_walk[j];
    a_j = j;
    if constexpr (GROUPED) a_b = wk.s;
    a_n = wk.n;
    a_base = wk.base;
    a_r = p.r[j];
  };
  auto load_walks = [&](int item) {  // returns this lane's
    DecodeWalk wk{0x7fffffff, 0, 0, 0u};
    if (lane < p.npat) wk = walk[(size_t)(item - first_item) * p.npat + lane];
    const DecodeHead hd = head[item - first_item];
    a_pos = hd.pos;
    a_b = hd.b;
    a_hk = item_of(p, item, tokens_of_item).hk;
    a_tiles = item == end.item ? end.tile : hd.tiles;
    a_walks = __ballot_sync(0xffffffffu, wk.n > 0);
    a_in = __ballot_sync(0xffffffffu, wk.heads & 1u);
    if (lane < kMaxPat) s_walk[lane] = wk;
    __syncwarp();
    return wk;
  };
  auto first_walk = [&]() {
    set_walk(a_walks != 0 ? __ffs(a_walks) - 1 : 0);
    a_k = 0;
  };
  // look up the pages of the next tile's rows
  auto look_up = [&]() {
    f_some = a_some;
    if (!f_some) return;
    const uint32_t k = a_k + row_l, n = (uint32_t)a_n;  // k may pass 2^31 in the last tile
    f_hk = a_hk;
    f_j = a_j;
    f_page = -1;
    f_meta = 0;
    const int x0 = (int)((uint32_t)a_base + a_k * (uint32_t)a_r);
    f_whole = a_r == 1 && a_k + kDecTile <= n && (x0 & 15) == 0;  // no page ends inside a half
    if (k < n) {
      f_x = x0 + row_l * a_r;
      f_page = p.geom.table[(size_t)a_b * p.geom.max_pages + (f_x >> p.geom.lp)];
    }
    if (MODE != kAnyPatterns || p.dense) {
      f_meta = k < n ? (GROUPED ? (uint32_t)f_x + 1 : 1u) : 0u;
    } else {
      // patterns that hold the row: low half; the one that walks it and all before: high half
      const int last = (int)((uint32_t)a_base + min(a_k + kDecTile - 1, n - 1) * (uint32_t)a_r);
      uint32_t held = 1u << a_j;
      for (int i = 0; i < p.npat; ++i) {
        const int si = s_walk[i].s;
        if (i == a_j || last < si) continue;
        if (f_x >= si && divides(p, i, a_pos - f_x)) held |= 1u << i;
      }
      const uint32_t upto = (2u << a_j) - 1;
      if constexpr (HEADS == 1) {  // how often the row counts
        const uint32_t u = held & a_in;
        f_meta = k < n && (u & upto) == (1u << a_j) ? __popc(u) : 0;
      } else {
        f_meta = k < n ? held | upto << 16 : 0u;
      }
    }
    a_k += kDecTile;
    if (--a_tiles == 0) {
      a_some = a_item != end.item && (a_item + 1 != end.item || end.tile != 0);
      if (a_some) {
        __syncwarp();
        load_walks(++a_item);
        first_walk();
      }
    } else if (a_k >= n) {
      a_k = 0;
      set_walk(max(__ffs(a_walks & ~((2u << a_j) - 1)) - 1, 0));
    }
  };
  constexpr int KQ = D / 64, VW = D / 32;  // 16-byte pieces of a K row, words of a V row, that a lane holds
  const uint8_t* const base_k = p.codes[0] + c * 16;
  const uint8_t* const base_v = p.codes[1] + g * (D / 8);
  uint32_t row = 0, row2 = 0, meta_l = 0;  // this lane's row of the cache, and what f_meta said of it
  float ks_l = 0.f, vs_l = 0.f;
  int walk_l = 0;
  bool whole = false, any = false;
  uint4 kr[4][KQ];
  uint32_t vr[8][VW];
  // take the looked-up tile: its rows' places and scales
  auto resolve = [&]() {
    bool in = f_meta != 0;
    if (in && (unsigned)f_page >= (unsigned)p.geom.pages) {
      p.geom.err.raise(kErrBadPage);
      in = false;
    }
    const uint32_t blk = in ? (uint32_t)f_page * (uint32_t)p.geom.Hkv + (uint32_t)f_hk : 0u;
    ks_l = vs_l = 1.f;
    if (in) {
      ks_l = p.scale[0][blk];
      vs_l = p.scale[1][blk];
    }
    meta_l = in ? f_meta : 0u;
    walk_l = f_j;
    row = in ? (blk << p.geom.lp) + (uint32_t)(f_x & pmask) : 0u;
    const uint32_t ins = __ballot_sync(0xffffffffu, in);
    any = ins != 0;
    whole = f_whole && ins == 0xffffffffu;
    if (whole) {  // two stretches of 16 rows: their first rows are lane 0's and, in slot 2, lane 2's
      row2 = __shfl_sync(0xffffffffu, row, 2);
      row = __shfl_sync(0xffffffffu, row, 0);
    } else {
      // a row that does not count stands for one that does: its codes are finite
      const uint32_t other = __shfl_sync(0xffffffffu, row, any ? __ffs(ins) - 1 : 0);
      if (!in) row = other;
    }
  };
  auto load_k = [&]() {
    if (whole) {
      const uint8_t* const half[2] = {base_k + (size_t)(row + (uint32_t)g) * D, base_k + (size_t)(row2 + (uint32_t)g) * D};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < KQ; ++q) kr[i][q] = load_codes16(half[i >> 1] + (i & 1) * 8 * D + q * 64);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // rows of slot i, row group g
        const uint8_t* src = base_k + (size_t)__shfl_sync(0xffffffffu, row, (lane & 28) | i) * D;
#pragma unroll
        for (int q = 0; q < KQ; ++q) kr[i][q] = load_codes16(src + q * 64);
      }
    }
  };
  auto load_v = [&]() {
    const uint8_t* const half[2] = {base_v + (size_t)(row + 2u * (uint32_t)c) * D, base_v + (size_t)(row2 + 2u * (uint32_t)c) * D};
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // rows of slot i / 2, row groups 2 c and 2 c + 1
      const uint8_t* src = half[i >> 2] + ((i >> 1) & 1) * 8 * D + (i & 1) * D;
      if (!whole) src = base_v + (size_t)__shfl_sync(0xffffffffu, row, 8 * c + 4 * (i & 1) + (i >> 1)) * D;
      if constexpr (D == 128) {
        const uint4 u = load_codes16(src);
        vr[i][0] = u.x, vr[i][1] = u.y, vr[i][2] = u.z, vr[i][3] = u.w;
      } else {
        const uint2 u = load_codes8(src);
        vr[i][0] = u.x, vr[i][1] = u.y;
      }
    }
  };

  // ---- the item in hand
  int tiles;                 // its tiles from here on, in the range
  float acc[MT][NB][4];
  float m[2 * NB], mv[2 * NB], l[2 * NB], fac[2 * NB];  // of columns nb * 8 + 2 c + e
  uint32_t in_pat[2 * NB];   // walks that each of the lane's columns takes part in
  int upto_pos[2 * NB];      // and their tokens' positions (p.tokens > 1)
  uint2 raw[NB][MT];  // q of head nb * 8 + g mod HW
  auto load_q = [&](int item) {
    const DecodeItem it = item_of(p, item, tokens_of_item);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int hl = nb * 8 + (g & (HW - 1));
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int d0 = (k >> 2) * 64 + c * 16 + (k & 3) * 4;
        raw[nb][k] = hl < it.nh ? *reinterpret_cast<const uint2*>(p.q + (long long)token_of(p, it, hl, tokens_of_item) * p.q_stride +
                                                                  head_of(p, it, hl, tokens_of_item) * D + d0)
                                : make_uint2(0, 0);
      }
    }
  };
  auto begin_item = [&](int item) {
    tiles = item == end.item ? end.tile : head[item - first_item].tiles;
    const uint32_t heads = lane < p.npat ? walk[(size_t)(item - first_item) * p.npat + lane].heads : 0u;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      // q lifted by a power of two to [2^13, 2^14): exact in fp16
      // (elements under 2^-37 of the largest are cut)
      uint32_t big = 0;
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        big = max(max(big, raw[nb][k].x & 0x7fffu), (raw[nb][k].x >> 16) & 0x7fffu);
        big = max(max(big, raw[nb][k].y & 0x7fffu), (raw[nb][k].y >> 16) & 0x7fffu);
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // exponent of the largest, from -96 on: every bf16 number is a multiple of 2^-133, which the
      // lift by 2^109 takes to fp16's smallest, and its inverse times qk_scale stays a normal number
      const int e = max((int)(big >> 7) - 127, -96);
      // 2^(13 - e) in two factors that fp32 holds
      const int up = 13 - e, u1 = up / 2, u2 = up - u1;
      const float f1 = __uint_as_float((uint32_t)(u1 + 127) << 23), f2 = __uint_as_float((uint32_t)(u2 + 127) << 23);
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const __half2 a = __floats2half2_rn(__uint_as_float(raw[nb][k].x << 16) * f1 * f2,
                                            __uint_as_float(raw[nb][k].x & 0xffff0000u) * f1 * f2);
        const __half2 b = __floats2half2_rn(__uint_as_float(raw[nb][k].y << 16) * f1 * f2,
                                            __uint_as_float(raw[nb][k].y & 0xffff0000u) * f1 * f2);
        qf[(nb * MT + k) * 32] = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
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
        upto_pos[2 * nb + e2] = 0;
        if constexpr (GROUPED) {
          const DecodeItem it = item_of(p, item, tokens_of_item);
          upto_pos[2 * nb + e2] = p.pos[token_of(p, it, min(nb * 8 + 2 * c + e2, it.nh - 1), tokens_of_item)];
        }
      }
      if constexpr (HEADS > 1) {
#pragma unroll
        for (int k = 0; k < HW; ++k) {
          const uint32_t b = __ballot_sync(0xffffffffu, heads >> (nb * 8 + k) & 1u);
          if (((2 * c) & (HW - 1)) == (k & ~1)) in_pat[2 * nb + (k & 1)] = b;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[mt][nb][k] = 0.f;
    }
  };

  // where a lane's sums of one of its heads lie: d = g (D / 8) + 0 .. D / 8 - 1
  auto sum_of = [&](int nb, int e, int k) { return acc[k >> 1][nb][(k & 1) * 2 + e]; };

  // The item is done here (slot < 0: this warp had all of it), or a partial of it goes to the slot.
  auto end_item = [&](int item, int slot) {
    const DecodeItem it = item_of(p, item, tokens_of_item);
    float* const dst = part + max(slot, 0) * slot_stride;
#pragma unroll
    for (int i = 0; i < 2 * NB; ++i) {
#pragma unroll
      for (int s = HW <= 2 ? 1 : HW == 4 ? 2 : 4; s < 32; s <<= 1)
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], s);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int i = 2 * nb + e, hl = nb * 8 + 2 * c + e;
        if (hl >= it.nh) continue;
        if (slot < 0) {
          const float f = final_factor(m[i], mv[i], l[i]);
          const size_t oi = place_of(p, it, hl, tokens_of_item);
          uint32_t o[D / 16];
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            // no row: 0, whatever the sums hold
            const __nv_bfloat162 v = l[i] == 0.f ? __floats2bfloat162_rn(0.f, 0.f)
                : __floats2bfloat162_rn(sum_of(nb, e, 2 * k) * f, sum_of(nb, e, 2 * k + 1) * f);
            o[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
          uint4* to = reinterpret_cast<uint4*>(p.out + oi * D + g * (D / 8));
#pragma unroll
          for (int k = 0; k < D / 64; ++k)
            to[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (g == 0 && p.lse != nullptr) p.lse[oi] = final_lse(m[i], l[i]);
        } else {
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            *reinterpret_cast<float4*>(dst + hl * D + g * (D / 8) + 4 * k) =
                make_float4(sum_of(nb, e, 4 * k), sum_of(nb, e, 4 * k + 1), sum_of(nb, e, 4 * k + 2),
                            sum_of(nb, e, 4 * k + 3));
          if (g == 0)
            *reinterpret_cast<float4*>(dst + p.part_heads * D + hl * 4) = make_float4(m[i], mv[i], l[i], 1.f);
        }
      }
  };

  // ---- start: the walk that the first tile belongs to
  load_q(a_item);
  const DecodeWalk wk = load_walks(a_item);
  a_tiles -= rg.tile;
  if (rg.tile == 0) {
    first_walk();
  } else {
    uint32_t past = ((uint32_t)wk.n + kDecTile - 1) / kDecTile;  // tiles of walks up to this lane's
#pragma unroll
    for (int s = 1; s < kMaxPat; s <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, past, s);
      if (lane >= s) past += y;
    }
    const int j = __popc(__ballot_sync(0xffffffffu, lane < p.npat && (uint32_t)rg.tile >= past));
    const uint32_t before = j > 0 ? __shfl_sync(0xffffffffu, past, j - 1) : 0u;
    set_walk(j);
    a_k = ((uint32_t)rg.tile - before) * kDecTile;
  }
  look_up();
  int item = rg.item;
  bool from_start = rg.tile == 0;
  begin_item(item);  // while the first tile's page numbers come
  tiles -= rg.tile;
  resolve();
  load_k();
  load_v();
  look_up();
  for (bool more = true; more;) {
    // ---- scores: block rb's rows g and g + 8, columns nb * 8 + 2 c and + 1
    float sc[2][NB][4];
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[rb][nb][k] = 0.f;
#pragma unroll
    for (int q = 0; q < KQ; ++q)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint2 qk[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) qk[nb] = qf[(nb * MT + q * 4 + k) * 32];
#pragma unroll
        for (int rb = 0; rb < 2; ++rb) {
          const uint4 ka = kr[2 * rb][q], kb = kr[2 * rb + 1][q];
          const uint32_t wa = k == 0 ? ka.x : k == 1 ? ka.y : k == 2 ? ka.z : ka.w;
          const uint32_t wb = k == 0 ? kb.x : k == 1 ? kb.y : k == 2 ? kb.z : kb.w;
          uint32_t a0, a1, a2, a3;
          codes_to_half<FMT>(wa, a0, a2);
          codes_to_half<FMT>(wb, a1, a3);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_16816(sc[rb][nb], a0, a1, a2, a3, qk[nb].x, qk[nb].y);
        }
      }
    // ---- what the softmax needs of the lane's rows (slots first_slot ..); then the next tile
    float ks[VR], lv[VR];
    uint32_t meta[VR];
    const bool some = any;
    const int walk_j = walk_l;
    {
      const float lv_l = fast_log2(vs_l);
#pragma unroll
      for (int v = 0; v < VR; ++v) {
        ks[v] = ks_l, lv[v] = lv_l, meta[v] = meta_l;
        const int from = (lane & 28) | (first_slot + v);
        // a half of a whole tile has one scale, and a lane of two rows has them in one half
        if (VR > 1 && (!whole || (VR == 4 && row >> p.geom.lp != row2 >> p.geom.lp))) {
          ks[v] = __shfl_sync(0xffffffffu, ks_l, from);
          lv[v] = __shfl_sync(0xffffffffu, lv_l, from);
        }
        if (VR > 1 && (GROUPED || !(whole && (MODE == kDense || p.dense)))) meta[v] = __shfl_sync(0xffffffffu, meta_l, from);
      }
    }
    more = f_some;
    if (more) {
      resolve();
      load_k();
      look_up();
    }
    // ---- softmax weights
    float s1[VR][NB][VE], s2[VR][NB][VE], cnt[VR][NB][VE];
    bool raise = false;
#pragma unroll
    for (int v = 0; v < VR; ++v) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int i = 2 * nb + e;
          float x;
          if constexpr (VR == 1) {
            const float x0 = c & 1 ? sc[0][nb][2 + e] : sc[0][nb][e];
            const float x1 = c & 1 ? sc[1][nb][2 + e] : sc[1][nb][e];
            x = c & 2 ? x1 : x0;
          } else if constexpr (VR == 2) {
            x = c & 2 ? sc[1][nb][2 * v + e] : sc[0][nb][2 * v + e];
          } else {
            x = sc[v >> 1][nb][(v & 1) * 2 + e];
          }
          float s, t;
          cnt[v][nb][e] = 1.f;
          if constexpr (MODE == kDense) {
            // chosen, not added: a row that is not there has a product of any kind (its query or a
            // substitute's codes may be NaN), but a finite lv
            s = meta[v] != 0 ? x * (fac[i] * ks[v]) : -INFINITY;
            t = s + lv[v];
          } else {
            bool ok = meta[v] != 0;
            if constexpr (GROUPED) {
              ok = ok && (int)(meta[v] - 1) <= upto_pos[i] && (in_pat[i] >> walk_j & 1u);
            } else if constexpr (HEADS == 1) {
              cnt[v][nb][e] = (float)(meta[v] & 31u);
            } else if (!p.dense) {
              const uint32_t u = meta[v] & in_pat[i], upto = meta[v] >> 16;
              ok = ok && (u & upto) == (upto ^ (upto >> 1));
              cnt[v][nb][e] = (float)__popc(u);
            }
            s = ok ? x * (fac[i] * ks[v]) : -INFINITY;
            t = ok ? s + lv[v] : -INFINITY;
          }
          s1[v][nb][e] = s;
          s2[v][nb][e] = t;
          raise = raise || s > m[i] + kMaxSlack || t > mv[i] + kMaxSlack;
        }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int i = 2 * nb + e;
          float a = s1[0][nb][e], b = s2[0][nb][e];
#pragma unroll
          for (int v = 1; v < VR; ++v) {
            a = fmaxf(a, s1[v][nb][e]);
            b = fmaxf(b, s2[v][nb][e]);
          }
#pragma unroll
          for (int s = HW <= 2 ? 1 : HW == 4 ? 2 : 4; s < 32; s <<= 1) {
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
    uint32_t pf[2][NB][2];  // P^T fragments of block rb
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t tr[VR];
#pragma unroll
      for (int v = 0; v < VR; ++v) {
        float pv[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int i = 2 * nb + e;
          const float p1 = fast_exp2(s1[v][nb][e] - m[i]), p2 = fast_exp2(s2[v][nb][e] - (mv[i] - kPBias));
          l[i] += MODE == kAnyPatterns ? p1 * cnt[v][nb][e] : p1;
          pv[e] = MODE == kAnyPatterns ? p2 * cnt[v][nb][e] : p2;
        }
        const __half2 h2 = __floats2half2_rn(pv[0], pv[1]);
        tr[v] = transpose8x8(*reinterpret_cast<const uint32_t*>(&h2));
      }
      // the transpose has column 2 c + e of lane group c in row group 2 c + e: the heads of
      // other slots go to row groups 0 .. HW - 1; the columns past them are not used
      if constexpr (VR == 1) {
        pf[0][nb][0] = tr[0];
        pf[0][nb][1] = __shfl_xor_sync(0xffffffffu, tr[0], 8);
        pf[1][nb][0] = __shfl_xor_sync(0xffffffffu, tr[0], 16);
        pf[1][nb][1] = __shfl_xor_sync(0xffffffffu, tr[0], 24);
      } else if constexpr (VR == 2) {
        pf[0][nb][0] = tr[0];
        pf[0][nb][1] = tr[1];
        pf[1][nb][0] = __shfl_xor_sync(0xffffffffu, tr[0], 16);
        pf[1][nb][1] = __shfl_xor_sync(0xffffffffu, tr[1], 16);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) pf[v >> 1][nb][v & 1] = tr[v];
      }
    }
    // ---- O^T += V^T P^T
    if (some) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb)
#pragma unroll
        for (int k = 0; k < VW; ++k)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            codes_to_half<FMT>(__byte_perm(vr[rb * 4][k], vr[rb * 4 + 1][k], sel), a0, a1);
            codes_to_half<FMT>(__byte_perm(vr[rb * 4 + 2][k], vr[rb * 4 + 3][k], sel), a2, a3);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_16816(acc[2 * k + half][nb], a0, a1, a2, a3, pf[rb][nb][0], pf[rb][nb][1]);
          }
    }
    if (more) load_v();
    if (--tiles == 0) {
      end_item(item, !from_start ? 0 : item == end.item ? 1 : -1);
      if (more) {
        from_start = true;
        load_q(++item);
        begin_item(item);
      }
    }
  }
}

template <int D, int HEADS, int FMT, int MODE>
__global__ void __launch_bounds__(kDecWarps * 32, decode_blocks_per_sm(D, HEADS, MODE == kGrouped))
    decode_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ uint2 s_q[kDecWarps][(HEADS + 7) / 8 * D / 16 * 32];
  __shared__ DecodeWalk s_walk[kDecWarps][kMaxPat];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // neighbouring warps of the sequence on different SMs: few ranges spread over all
  const int wi = warp * (int)gridDim.x + (int)blockIdx.x;
  grid_dependency_wait();
  const DecodeRange rg = p.range[wi], end = p.range[wi + 1];
  grid_dependency_release();
  if (rg.item == end.item && rg.tile == end.tile) return;
  decode_range<D, HEADS, FMT, MODE>(p, rg, end, p.head, p.walk, 0, p.part + (size_t)wi * 2 * p.part_stride,
                                       p.part_stride, s_q[warp] + lane, s_walk[warp]);
}

__device__ __forceinline__ void add_scaled(float4& a, const float4& x, float f) {
  a.x += x.x * f;
  a.y += x.y * f;
  a.z += x.z * f;
  a.w += x.w * f;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
  return x;
}
// Elements 4 col .. 4 col + 3 of a head's result.
__device__ __forceinline__ void store_joined(const DecodeParams& p, int D, size_t oi, int col, float4 a, float M,
                                             float MV, float L) {
  const float f = final_factor(M, MV, L);
  if (L == 0.f) a = make_float4(0.f, 0.f, 0.f, 0.f);  // no row: 0, whatever the sums hold
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * f, a.y * f), hi = __floats2bfloat162_rn(a.z * f, a.w * f);
  *reinterpret_cast<uint2*>(p.out + oi * D + col * 4) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  if (col == 0 && p.lse != nullptr) p.lse[oi] = final_lse(M, L);
}

// ---------------------------------------------------------------------------
// Few or short items, in one launch. A team has an item: a warp (p.team = 0), or
// the 8 warps each of p.team blocks of a cluster. It describes the item, its
// warps take equal shares of the tiles, and the partials come together in
// shared memory, the block's first and then the cluster's.
// ---------------------------------------------------------------------------
constexpr int kTeamBlocks = 8;        // most blocks of a team
constexpr int kTeamWarps = 8;         // warps of a block

template <int D, int HEADS, int FMT>
__global__ void __launch_bounds__(kTeamWarps * 32, D == 64 && HEADS <= 8 ? 2 : 1)
    decode_team_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ float4 s_dyn[];       // partials of the warps, then the block's
  __shared__ uint2 s_q[kTeamWarps][(HEADS + 7) / 8 * D / 16 * 32];
  __shared__ DecodeWalk s_walk[kTeamWarps][kMaxPat], s_desc[kTeamWarps][kMaxPat];
  __shared__ DecodeHead s_head[kTeamWarps];
  float* const s_part = reinterpret_cast<float*>(s_dyn);
  float* const s_block = s_part + kTeamWarps * p.part_stride;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int stat = p.part_heads * D;      // where a partial's statistics begin
  const bool alone = p.team == 0;
  const int blocks = max(p.team, 1), rank = (int)blockIdx.x % blocks;
  const int item = alone ? (int)blockIdx.x * kTeamWarps + warp : (int)blockIdx.x / blocks;
  const int own = alone ? warp : 0;       // whose description it is
  grid_dependency_wait();
  grid_dependency_release();
  if (alone && item >= p.items) return;
  if (alone || warp == 0) describe_item(p, item, &s_head[own], s_desc[own]);
  if (alone) __syncwarp(); else __syncthreads();
  {
    DecodeRange rg{item, 0}, end{item + 1, 0};
    if (!alone) {
      const int k = warp * blocks + rank, n = blocks * kTeamWarps;
      const long long tiles = s_head[0].tiles;
      rg.tile = (int)(tiles * k / n);
      end = DecodeRange{item, (int)(tiles * (k + 1) / n)};
    }
    float* const part = s_part + warp * p.part_stride;
    if (alone || rg.tile < end.tile)
      decode_range<D, HEADS, FMT, kAnyPatterns>(p, rg, end, &s_head[own], s_desc[own], item, part, 0, s_q[warp] + lane,
                                         s_walk[warp]);
    else if (lane < p.part_heads)
      reinterpret_cast<float4*>(part + stat)[lane] = make_float4(kNoMax, kNoMax, 0.f, 0.f);
  }
  if (alone) return;
  __syncthreads();
  const DecodeItem it = item_of(p, item, p.tokens);
  const int pieces = it.nh * (D / 4);
  // element piece i of up to eight partials, the k-th one at part(k); those whose mark is 0 are not there
  auto join = [&](auto part, int n, int i, float& M, float& MV, float& L) {
    const int hl = i / (D / 4);
    float4 st[8], x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      st[k] = make_float4(kNoMax, kNoMax, 0.f, 0.f);
      if (k < n) {
        st[k] = *reinterpret_cast<const float4*>(part(k) + stat + hl * 4);
        x[k] = reinterpret_cast<const float4*>(part(k))[i];
      }
    }
    M = MV = kNoMax;
#pragma unroll
    for (int k = 0; k < 8; ++k) M = fmaxf(M, st[k].x), MV = fmaxf(MV, st[k].y);
    L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (st[k].w == 0.f) continue;
      L += st[k].z * exp2f(st[k].x - M);
      add_scaled(a, x[k], exp2f(st[k].y - MV));
    }
    return a;
  };
  static_assert(kTeamWarps <= 8 && kTeamBlocks <= 8, "join takes eight");
  for (int i = tid; i < pieces; i += kTeamWarps * 32) {
    float M, MV, L;
    reinterpret_cast<float4*>(s_block)[i] =
        join([&](int k) { return s_part + k * p.part_stride; }, kTeamWarps, i, M, MV, L);
    if (i % (D / 4) == 0) *reinterpret_cast<float4*>(s_block + stat + i / (D / 4) * 4) = make_float4(M, MV, L, 1.f);
  }
  cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  cluster.sync();
  for (int i = tid * blocks + rank; i < pieces; i += kTeamWarps * 32 * blocks) {
    float M, MV, L;
    const float4 a = join([&](int k) { return (const float*)cluster.map_shared_rank(s_block, k); }, blocks, i,
                          M, MV, L);
    const int hl = i / (D / 4);
    store_joined(p, D, place_of(p, it, hl, p.tokens), i % (D / 4), a, M, MV, L);
  }
  cluster.sync();  // no block ends while another reads its sums
}

// ---------------------------------------------------------------------------
// Join of cut items. An item that begins in warp w's range and goes on past it
// has its partials in slot 1 of w and in slot 0 of the warps behind it.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kJoinPart = 512;  // partials whose weights are held at a time
constexpr int kJoinShort = 32;  // most partials that one warp joins

// The partials of an item: the k-th one from range w on.
struct JoinParts {
  const float* first;
  const float* rest;  // partial k > 0 at rest + k step
  size_t step;
  __device__ JoinParts(const DecodeParams& p, int w)
      : first(p.part + ((size_t)w * 2 + 1) * p.part_stride),
        rest(p.part + (size_t)w * 2 * p.part_stride),
        step((size_t)2 * p.part_stride) {}
  __device__ const float* operator()(int k) const { return k == 0 ? first : rest + k * step; }
};

// One warp joins a column of up to kJoinShort partials.
template <int D>
__device__ __forceinline__ void join_short(const DecodeParams& p, const DecodeItem& it, int w, int n, int column) {
  constexpr int LANES = D / 4, ROWS = 32 / LANES;  // threads of a row, rows at a time
  constexpr int EAGER = 4;
  const int lane = threadIdx.x & 31, row = lane / LANES, col = lane % LANES;
  const JoinParts part(p, w);
  float4 st = make_float4(kNoMax, kNoMax, 0.f, 0.f);
  if (lane < n) st = *reinterpret_cast<const float4*>(part(lane) + p.part_heads * D + column * 4);
  float4 x[EAGER];  // the first rows come along with the statistics
#pragma unroll
  for (int i = 0; i < EAGER; ++i) {
    const int k = i * ROWS + row;
    if (k < n) x[i] = *reinterpret_cast<const float4*>(part(k) + column * D + col * 4);
  }
  const float M = warp_max(st.x), MV = warp_max(st.y);
  const float L = warp_sum(lane < n ? st.z * exp2f(st.x - M) : 0.f);
  const float f = exp2f(st.y - MV);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < EAGER; ++i) {
    const float fk = __shfl_sync(0xffffffffu, f, i * ROWS + row);
    if (i * ROWS + row < n) add_scaled(acc, x[i], fk);
  }
#pragma unroll 4
  for (int k0 = EAGER * ROWS; k0 < n; k0 += ROWS) {
    const int k = k0 + row;
    const float fk = __shfl_sync(0xffffffffu, f, k & 31);
    if (k < n) add_scaled(acc, *reinterpret_cast<const float4*>(part(k) + column * D + col * 4), fk);
  }
  if constexpr (LANES == 16) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, 16);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, 16);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, 16);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, 16);
  }
  if (row == 0) store_joined(p, D, place_of(p, it, column, p.tokens), col, acc, M, MV, L);
}

// A block joins a column of any number of partials; BATCH: rows of a thread under way at once.
template <int D, int BATCH>
__device__ __forceinline__ void join_long(const DecodeParams& p, const DecodeItem& it, int w, int n, int column) {
  constexpr int LANES = D / 4, STEP = kJoinThreads / LANES;
  constexpr int OWN = kJoinPart / kJoinThreads;
  __shared__ float s_l[kJoinPart], s_v[kJoinPart];
  __shared__ float s_top[kJoinWarps][2], s_sum;
  __shared__ float4 s_acc[STEP][LANES];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = tid / LANES, col = tid % LANES;
  const int so = p.part_heads * D + column * 4;
  const JoinParts part(p, w);
  // statistics of the first kJoinPart partials, and the first rows of sums, come along
  float4 st[OWN], x[BATCH];
  auto load_rows = [&](int base, int i0, int cnt) {
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = i0 + j * STEP;
      if (i < cnt) x[j] = *reinterpret_cast<const float4*>(part(base + i) + column * D + col * 4);
    }
  };
  float2 top = make_float2(kNoMax, kNoMax);
#pragma unroll
  for (int u = 0; u < OWN; ++u) {
    const int k = tid + u * kJoinThreads;
    st[u] = k < n ? *reinterpret_cast<const float4*>(part(k) + so) : make_float4(kNoMax, kNoMax, 0.f, 0.f);
  }
  load_rows(0, row, min(n, kJoinPart));
#pragma unroll
  for (int u = 0; u < OWN; ++u) top = make_float2(fmaxf(top.x, st[u].x), fmaxf(top.y, st[u].y));
  for (int k = kJoinPart + tid; k < n; k += kJoinThreads) {
    const float2 f = *reinterpret_cast<const float2*>(part(k) + so);
    top = make_float2(fmaxf(top.x, f.x), fmaxf(top.y, f.y));
  }
  float M = warp_max(top.x), MV = warp_max(top.y);
  if (lane == 0) s_top[warp][0] = M, s_top[warp][1] = MV;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    M = fmaxf(M, s_top[k][0]);
    MV = fmaxf(MV, s_top[k][1]);
  }
  // sums, in the partials' order
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < n; base += kJoinPart) {
    const int cnt = min(kJoinPart, n - base);
#pragma unroll
    for (int u = 0; u < OWN; ++u) {
      const int i = tid + u * kJoinThreads;
      if (base > 0 && i < cnt) st[u] = *reinterpret_cast<const float4*>(part(base + i) + so);
      if (i < cnt) {
        s_l[i] = st[u].z * exp2f(st[u].x - M);
        s_v[i] = exp2f(st[u].y - MV);
      }
    }
    __syncthreads();
    for (int i0 = row; i0 < cnt; i0 += STEP * BATCH) {
      if (base > 0 || i0 != row) load_rows(base, i0, cnt);
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (i0 + j * STEP < cnt) add_scaled(acc, x[j], s_v[i0 + j * STEP]);
    }
    if (warp == 0)
      for (int i = lane; i < cnt; i += 32) L += s_l[i];
    __syncthreads();
  }
  s_acc[row][col] = acc;
  if (warp == 0) {
    L = warp_sum(L);
    if (lane == 0) s_sum = L;
  }
  __syncthreads();
  if (tid < LANES) {
    float4 a = s_acc[0][tid];
#pragma unroll
    for (int k = 1; k < STEP; ++k) add_scaled(a, s_acc[k][tid], 1.f);
    store_joined(p, D, place_of(p, it, column, p.tokens), tid, a, M, MV, s_sum);
  }
}

// The ranges are there before a join kernel waits: it was let start after every block of the main
// one had waited for the plan. What other kernels left of them in L1 is passed over.
__device__ __forceinline__ DecodeRange range_of(const DecodeParams& p, int k) {
  const int2 x = __ldcg(reinterpret_cast<const int2*>(p.range + k));
  return DecodeRange{x.x, x.y};
}

// Few items: blockIdx.x is the item, whose columns are a warp's each when it has few partials, and
// else a block's each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 2) decode_join_items_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ int s_cnt[kJoinWarps][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, item = (int)blockIdx.x;
  int before = 0, in = 0;  // ranges that begin up to the item's beginning, and inside it
  for (int k = tid; k <= p.warps; k += kJoinThreads) {
    const DecodeRange r = range_of(p, k);
    before += r.item < item || (r.item == item && r.tile == 0);
    in += r.item == item && r.tile > 0;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  in = __reduce_add_sync(0xffffffffu, in);
  if (lane == 0) s_cnt[warp][0] = before, s_cnt[warp][1] = in;
  __syncthreads();
  before = in = 0;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) before += s_cnt[k][0], in += s_cnt[k][1];
  grid_dependency_wait();
  grid_dependency_release();
  const int w = before - 1, n = in + 1;
  if (n == 1) return;  // not cut
  const DecodeItem it = item_of(p, item, p.tokens);
  if (n <= kJoinShort) {
    const int column = (int)blockIdx.y * kJoinWarps + warp;
    if (column < it.nh) join_short<D>(p, it, w, n, column);
  } else if ((int)blockIdx.y < it.nh) {
    join_long<D, 8>(p, it, w, n, blockIdx.y);
  }
}

// Many items: block (x, y) has column y of the items that begin in ranges 8 x .. 8 x + 7, a warp
// each; one of more partials (no second one begins in eight ranges) is the whole block's.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) decode_join_ranges_kernel(const __grid_constant__ DecodeParams p) {
  __shared__ int s_long;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, column = blockIdx.y;
  const int w = (int)blockIdx.x * kJoinWarps + warp;
  if (tid == 0) s_long = -1;
  DecodeRange a{0, 0}, b{0, 0}, r{-1, 0};  // r: ranges w + 1 .., those that hold a part of the item
  if (w < p.warps) {
    a = range_of(p, w);
    b = range_of(p, w + 1);
    if (w + 1 + lane < p.warps) r = range_of(p, w + 1 + lane);
  }
  grid_dependency_wait();
  grid_dependency_release();
  __syncthreads();
  // an item begins in range w and goes on past it
  if (b.tile > 0 && (a.item != b.item || a.tile == 0)) {
    const DecodeItem it = item_of(p, b.item, p.tokens);
    const uint32_t held = __ballot_sync(0xffffffffu, r.item == b.item);
    if (column >= it.nh) {
    } else if (__popc(held) < kJoinShort) {
      join_short<D>(p, it, w, __popc(held) + 1, column);
    } else if (lane == 0) {
      s_long = w;
    }
  }
  __syncthreads();
  const int wl = s_long;
  if (wl < 0) return;
  const int item = range_of(p, wl + 1).item;
  int n = 1;
  for (int k = wl + 1 + tid;; k += kJoinThreads) {
    const int got = __syncthreads_count(k < p.warps && range_of(p, k).item == item);
    n += got;
    if (got < kJoinThreads) break;
  }
  join_long<D, 2>(p, item_of(p, item, p.tokens), wl, n, column);  // rare: registers for more blocks
}

}  // namespace dil
