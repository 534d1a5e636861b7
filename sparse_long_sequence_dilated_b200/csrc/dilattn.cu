// libdilattn: C-ABI entry points (validation, TMA descriptor set-up, launches).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "dilattn.h"
#include "common.cuh"
#include "fwd_tc.cuh"
#include "bwd_tc.cuh"
#include "simt.cuh"
#include "cache.cuh"
#include "decode.cuh"

namespace dil {

__device__ int g_dev_error;  // device-side error word (bounded waits that ran out)

// Self-test of the failure path: warp 0 waits on an mbarrier that nothing
// arrives on, with a limit of limit_ns; warp 1 waits on another one with the
// kernels' ordinary 4 s limit and must give up as soon as warp 0 has raised
// the CTA's abort flag. result[0], result[1]: 1 if the warp's wait completed
// (it must not), 0 if it gave up; result[2], result[3]: nanoseconds each
// warp waited.
__global__ void selftest_wait_kernel(ErrCtx err, unsigned long long limit_ns, int* result) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ volatile int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    const unsigned long long t0 = globaltimer_ns();
    const bool ok = warp == 0
        ? mbar_wait(smem_u32(&bars[0]), 0, &abort_flag, err, limit_ns)
        : mbar_wait(smem_u32(&bars[1]), 0, &abort_flag, err);
    result[warp] = ok ? 1 : 0;
    result[2 + warp] = (int)min(globaltimer_ns() - t0, 2000000000ull);
  }
}

namespace {

thread_local char g_last_error[512] = "";

// Launch tags for the device error word (see ErrCtx): 1 .. 2^23 - 1, cycling.
std::atomic<unsigned> g_launch_tag{0};
int next_tag() { return (int)(g_launch_tag.fetch_add(1u) % 0x7FFFFFu) + 1; }


int cuda_fail(cudaError_t e, const char* what) {
  snprintf(g_last_error, sizeof(g_last_error), "%s: %s (%d)", what, cudaGetErrorString(e),
           (int)e);
  return DILATTN_ERR_CUDA;
}

thread_local cudaEvent_t g_trace_begin = nullptr;
thread_local cudaEvent_t g_trace_end = nullptr;

int trace_mark(cudaEvent_t ev, cudaStream_t stream) {
  if (ev == nullptr) return DILATTN_OK;
  cudaError_t e = cudaEventRecord(ev, stream);
  return e == cudaSuccess ? DILATTN_OK : cuda_fail(e, "cudaEventRecord");
}

// ------------------------------------------------------------------ device state
struct DeviceState {
  bool init = false;
  bool arch_ok = false;
  int* err_word = nullptr;
  int num_sms = 0;
  int dev = 0;
  cudaMemPool_t pool = nullptr;  // the forward's scratch pool, created on first use
};

std::mutex g_mu;
std::map<int, DeviceState> g_devices;

int device_state(DeviceState** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceState& st = g_devices[dev];
  st.dev = dev;
  if (!st.init) {
    int major = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    st.arch_ok = (major == 10);
    if (st.arch_ok) {
      e = cudaDeviceGetAttribute(&st.num_sms, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
      e = cudaGetSymbolAddress(reinterpret_cast<void**>(&st.err_word), g_dev_error);
      if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress");
      e = cudaFuncSetAttribute(fwd_tile_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               FwdCfg<64>::SMEM_BYTES);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
      e = cudaFuncSetAttribute(fwd_tile_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               FwdCfg<128>::SMEM_BYTES);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
      e = cudaFuncSetAttribute(fwd_tile_kernel<128, true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               FwdCfg<128, true>::SMEM_BYTES);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
      e = cudaFuncSetAttribute(bwd_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               BwdCfg::SMEM_BYTES);
      if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
    }
    st.init = true;
  }
  if (!st.arch_ok) return DILATTN_ERR_UNSUPPORTED;
  *out = &st;
  return DILATTN_OK;
}

// Stream-ordered memory pool of the device for the forward's scratch. Freed
// blocks stay in the pool (release threshold: never), so after the first call
// of a given size the forward maps no new memory.
int scratch_pool(DeviceState* st, cudaMemPool_t* out) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (st->pool == nullptr) {
    cudaMemPoolProps props;
    memset(&props, 0, sizeof(props));
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = st->dev;
    cudaMemPool_t pool = nullptr;
    cudaError_t e = cudaMemPoolCreate(&pool, &props);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemPoolCreate");
    uint64_t keep = ~0ull;
    e = cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemPoolSetAttribute");
    st->pool = pool;
  }
  *out = st->pool;
  return DILATTN_OK;
}

// ------------------------------------------------------------------ TMA descriptors
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

int get_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) {
    snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled unavailable");
    return DILATTN_ERR_CUDA;
  }
  return DILATTN_OK;
}

// Strided view of a [B][N][H][d] tensor (bf16, or fp32 when f32 is set) that
// gathers every r-th row, with the tensor's own base address: dims
// {d, H, P, M, B}, byte strides {e d, e H d, e H d r, e H d N} for element
// size e, so element (c, h, ph, m, b) is row ph + m*r of batch b. The main
// view has P = r phases and M = floor(N/r) rows; the tail view has
// P = N mod r and M = floor(N/r) + 1. Either way every in-bounds coordinate is
// a row below N; loads read zeros and stores/reduces skip rows past it. Box:
// 128 bytes of columns (128-byte swizzle) x box_rows rows (128, or 32 for the
// backward's per-warp reduce-adds).
using MapKey = std::tuple<const void*, int, int, int, int, int, int, int, int>;
std::mutex g_map_mu;
std::map<MapKey, CUtensorMap> g_maps;

int strided_map(const void* ptr, int B, int N, int H, int d, int r, int tail, CUtensorMap* out,
                int f32 = 0, int box_rows = BM) {
  const long long nfloor = N / r;
  const int nmod = N % r;
  if ((tail && nmod == 0) || (!tail && nfloor == 0)) {
    memset(out, 0, sizeof(*out));  // a view no tile of this problem can address
    return DILATTN_OK;
  }
  MapKey key{ptr, B, N, H, d, r, tail, f32, box_rows};
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    auto it = g_maps.find(key);
    if (it != g_maps.end()) {
      *out = it->second;
      return DILATTN_OK;
    }
  }
  int rc = get_encoder();
  if (rc != DILATTN_OK) return rc;
  const int esz = f32 == 1 ? 4 : f32 == 3 ? 1 : 2;  // f32: 0 bf16, 1 fp32, 2 fp16, 3 e4m3
  const long long rowb = (long long)H * d * esz;
  cuuint64_t dims[5] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)(tail ? nmod : r),
                        (cuuint64_t)(tail ? nfloor + 1 : nfloor), (cuuint64_t)B};
  cuuint64_t strides[4] = {(cuuint64_t)d * esz, (cuuint64_t)rowb, (cuuint64_t)(rowb * r),
                           (cuuint64_t)(rowb * N)};
  cuuint32_t box[5] = {(cuuint32_t)(128 / esz), 1, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUtensorMap m;
  const CUtensorMapDataType dt = f32 == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : f32 == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : f32 == 3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUresult cr = g_encode(&m, dt, 5, const_cast<void*>(ptr), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) {
    snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed (%d)", (int)cr);
    return DILATTN_ERR_CUDA;
  }
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    if (g_maps.size() > 4096) g_maps.clear();
    g_maps[key] = m;
  }
  *out = m;
  return DILATTN_OK;
}

// View of a gathered dilated buffer [ranks][B][rank_rows][H][d] bf16 whose
// row j of head h is dilated row j of that head's segment: dims
// {d, H, rank_rows, ranks, B}; a box of box_rows (64 or 128) rows never
// crosses a rank's block (rank_rows is a multiple of 128).
int gathered_map(const void* ptr, int B, int H, int d, int rank_rows, int ranks, CUtensorMap* out,
                 int box_rows = BM) {
  MapKey key{ptr, B, rank_rows, H, d, -ranks, 2, 0, box_rows};
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    auto it = g_maps.find(key);
    if (it != g_maps.end()) {
      *out = it->second;
      return DILATTN_OK;
    }
  }
  int rc = get_encoder();
  if (rc != DILATTN_OK) return rc;
  const cuuint64_t rowb = (cuuint64_t)H * d * 2;
  cuuint64_t dims[5] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rank_rows, (cuuint64_t)ranks,
                        (cuuint64_t)B};
  cuuint64_t strides[4] = {(cuuint64_t)d * 2, rowb, rowb * rank_rows * B, rowb * rank_rows};
  cuuint32_t box[5] = {64, 1, (cuuint32_t)box_rows, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUtensorMap m;
  CUresult cr = g_encode(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) {
    snprintf(g_last_error, sizeof(g_last_error), "cuTensorMapEncodeTiled failed (%d)", (int)cr);
    return DILATTN_ERR_CUDA;
  }
  {
    std::lock_guard<std::mutex> lk(g_map_mu);
    if (g_maps.size() > 4096) g_maps.clear();
    g_maps[key] = m;
  }
  *out = m;
  return DILATTN_OK;
}

// One sequence-parallel rank's per-pattern inputs (see FwdParams): patterns
// with kv_rows > 0 take K and V from the gathered buffers kg, vg.
struct SeqParPlan {
  int kv_rows[kMaxPat];
  int kv_rank_rows[kMaxPat];
  int ranks[kMaxPat];
  int toff[kMaxPat];
  const void* kg[kMaxPat];
  const void* vg[kMaxPat];
};

// ------------------------------------------------------------------ validation
int check_shape(int B, int N, int H, int d, const int* w, const int* r, int npat, int causal) {
  if (B < 1 || N < 1 || H < 1 || d < 1) return DILATTN_ERR_INVALID_ARG;
  if (npat < 1 || npat > DILATTN_MAX_PATTERNS || w == nullptr || r == nullptr)
    return DILATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return DILATTN_ERR_INVALID_ARG;
  const double elems = (double)B * N * H * d;
  if (elems >= 1099511627776.0) return DILATTN_ERR_INVALID_ARG;
  for (int i = 0; i < npat; ++i) {
    if (w[i] < 1 || r[i] < 1) return DILATTN_ERR_INVALID_ARG;
    if ((double)r[i] * H * d * 4 >= 1099511627776.0) return DILATTN_ERR_INVALID_ARG;
  }
  return DILATTN_OK;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const char* x = (const char*)a;
  const char* y = (const char*)b;
  return x < y + bn && y < x + an;
}

// Pattern geometry and partial-buffer layout. Pattern `skip` (the merging
// pattern, or -1) stores no partials and gets no rows. Returns the partial rows.
// Argument checks shared by the forward entry points.
int check_fwd_args(const void* q, const void* k, const void* v, const void* out, const float* lse,
                   int B, int N, int H, int d, const int* w, const int* r, int npat, int causal) {
  int rc = check_shape(B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return DILATTN_ERR_INVALID_ARG;
  if (lse != nullptr && !aligned16(lse)) return DILATTN_ERR_INVALID_ARG;
  const size_t tb = (size_t)B * N * H * d * 2;
  if (overlaps(out, tb, q, tb) || overlaps(out, tb, k, tb) || overlaps(out, tb, v, tb))
    return DILATTN_ERR_INVALID_ARG;
  if (lse != nullptr) {
    const size_t lb = (size_t)B * H * N * 4;
    if (overlaps(lse, lb, q, tb) || overlaps(lse, lb, k, tb) || overlaps(lse, lb, v, tb) ||
        overlaps(lse, lb, out, tb))
      return DILATTN_ERR_INVALID_ARG;
  }
  if (d != 64 && d != 128) return DILATTN_ERR_UNSUPPORTED;
  return DILATTN_OK;
}

long long make_geoms(int B, int N, int H, const int* w, const int* r, int npat,
                     PatternGeom* geo, int skip = -1) {
  long long rows = 0;
  for (int i = 0; i < npat; ++i) {
    PatternGeom& g = geo[i];
    g.w = w[i];
    g.r = r[i];
    divisor_magic((uint32_t)w[i], g.w_mul, g.w_sh);
    divisor_magic((uint32_t)r[i], g.r_mul, g.r_sh);
    g.nseg = (int)(((long long)N + w[i] - 1) / w[i]);
    const long long span = std::min<long long>(w[i], N);
    g.nmax = (int)((span + r[i] - 1) / r[i]);
    g.ntiles = (g.nmax + BM - 1) / BM;
    g.pstride = g.ntiles * BM;
    g.nmod = N % r[i];
    g.part_base = rows;
    if (i != skip) rows += (long long)B * H * g.nseg * g.pstride;
  }
  return rows;
}

// The merging pattern: one with r = 1 keeps every row of every head, so its
// tiles can finish the merge of all patterns. The shortest such pattern is
// taken (its tiles are the shortest, which keeps the end of the launch short).
int pick_merger(const int* w, const int* r, int npat) {
  int m = -1;
  for (int i = 0; i < npat; ++i)
    if (r[i] == 1 && (m < 0 || w[i] < w[m])) m = i;
  return m;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Longest-first unit order for the tile kernels (see Sched).
long long make_schedule(const PatternGeom* pat, int npat, int B, int H, Sched& sc,
                        unsigned include = 0xffffffffu) {
  std::vector<int> order;
  for (int i = 0; i < npat; ++i)
    if (include >> i & 1u) order.push_back(i);
  const int nsel = (int)order.size();
  memset(&sc, 0, sizeof(sc));
  if (nsel == 0) return 0;
  std::stable_sort(order.begin(), order.end(),
                   [&](int a, int b) { return pat[a].ntiles > pat[b].ntiles; });
  std::vector<int> vals;
  for (int i : order)
    if (vals.empty() || vals.back() != pat[i].ntiles) vals.push_back(pat[i].ntiles);
  for (int i = 0; i < nsel; ++i) sc.order[i] = order[i];
  sc.nband = (int)vals.size();
  sc.start[0] = 0;
  for (int j = 0; j < sc.nband; ++j) {
    const int lo = j + 1 < sc.nband ? vals[j + 1] : 0;
    sc.nt[j] = vals[j];
    int act = 0;
    long long per = 0;
    for (int a = 0; a < nsel; ++a) {
      if (pat[order[a]].ntiles >= vals[j]) {
        ++act;
        per += (long long)pat[order[a]].nseg * B * H;
      }
    }
    sc.npat_active[j] = act;
    sc.per_level[j] = per;
    sc.start[j + 1] = sc.start[j] + (long long)(vals[j] - lo) * per;
  }
  sc.nt[sc.nband] = 0;
  return sc.start[sc.nband];
}

// Forward scratch: [rows][d] fp32 partial outputs, [rows] fp32 partial lse,
// one flag per 128-row block of partials, and the ticket counter.
struct FwdScratch {
  size_t o_bytes, lse_bytes, flag_bytes;
  size_t total() const { return o_bytes + lse_bytes + flag_bytes; }
};
FwdScratch fwd_scratch_layout(long long rows, int d) {
  FwdScratch f;
  f.o_bytes = align256((size_t)rows * d * 4);
  f.lse_bytes = align256((size_t)rows * 4);
  f.flag_bytes = align256((size_t)(rows / BM + 1) * 4 + 8);  // flags, the ticket and done counters
  return f;
}

size_t fwd_scratch_bytes(int B, int N, int H, int d, const int* w, const int* r, int npat) {
  PatternGeom geo[kMaxPat];
  const long long rows = make_geoms(B, N, H, w, r, npat, geo, pick_merger(w, r, npat));
  return fwd_scratch_layout(rows, d).total();
}

// A named host-side range for profilers (NVTX; a no-op unless a tool is
// attached), around each launch sequence.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

template <int D, bool QK8 = false>
int launch_fwd(const void* q, const void* k, const void* v, void* out, void* out_res, float* lse,
               int B, int N, int H, const int* w, const int* r, int npat, int causal, void* ws,
               DeviceState* st, cudaStream_t stream, const SeqParPlan* sp = nullptr,
               float qk_scale = 1.f) {
  static_assert(sizeof(FwdParams) < 32000, "kernel parameter block too large");
  NvtxRange range(QK8 ? "dilattn forward (e4m3 q, k)" : sp != nullptr ? "dilattn forward (sequence-parallel rank)"
                                                                        : "dilattn forward");
  FwdParams p;
  memset(&p, 0, sizeof(p));
  p.npat = npat;
  p.B = B;
  p.N = N;
  p.H = H;
  p.causal = causal;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D) * (double)qk_scale);
  p.merger = pick_merger(w, r, npat);
  const long long rows = make_geoms(B, N, H, w, r, npat, p.pat, p.merger);
  const FwdScratch lay = fwd_scratch_layout(rows, D);
  char* wsb = reinterpret_cast<char*>(ws);
  p.part_o = reinterpret_cast<float*>(wsb);
  p.part_lse = reinterpret_cast<float*>(wsb + lay.o_bytes);
  p.flags = reinterpret_cast<int*>(wsb + lay.o_bytes + lay.lse_bytes);
  p.counter = p.flags + rows / BM + 1;
  p.done = p.counter + 1;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.out_res = reinterpret_cast<__nv_bfloat16*>(out_res);
  p.lse = lse;
  p.err = ErrCtx{st->err_word, next_tag()};
  for (int i = 0; i < npat; ++i) {
    const void* src[3] = {q, k, v};
    const int dtype[3] = {QK8 ? 3 : 0, QK8 ? 3 : 0, 0};
    CUtensorMap* dst[3] = {&p.tmq[i], &p.tmk[i], &p.tmv[i]};
    CUtensorMap* dst_t[3] = {&p.tmq_t[i], &p.tmk_t[i], &p.tmv_t[i]};
    // Q tiles are BM rows; K and V tiles the kernel's key-tile rows
    constexpr int kbn = FwdCfg<D, QK8>::BN;
    for (int j = 0; j < 3; ++j) {
      const int rows = j == 0 ? BM : kbn;
      int rc = strided_map(src[j], B, N, H, D, r[i], 0, dst[j], dtype[j], rows);
      if (rc == DILATTN_OK) rc = strided_map(src[j], B, N, H, D, r[i], 1, dst_t[j], dtype[j], rows);
      if (rc != DILATTN_OK) return rc;
    }
    if (sp != nullptr && sp->kv_rows[i] > 0) {
      p.kv_rows[i] = sp->kv_rows[i];
      p.kv_rank_rows[i] = sp->kv_rank_rows[i];
      p.toff[i] = sp->toff[i];
      int rc = gathered_map(sp->kg[i], B, H, D, sp->kv_rank_rows[i], sp->ranks[i], &p.tmk[i], kbn);
      if (rc == DILATTN_OK)
        rc = gathered_map(sp->vg[i], B, H, D, sp->kv_rank_rows[i], sp->ranks[i], &p.tmv[i], kbn);
      if (rc != DILATTN_OK) return rc;
    }
  }
  const unsigned all = (1u << npat) - 1u;
  const unsigned mbit = p.merger >= 0 ? (1u << p.merger) : 0u;
  p.units_p = make_schedule(p.pat, npat, B, H, p.sched, all & ~mbit);
  const long long units_m = mbit ? make_schedule(p.pat, npat, B, H, p.sched_m, mbit) : 0;
  const long long units = p.units_p + units_m;
  if (units > 0x7fffffffLL) return DILATTN_ERR_UNSUPPORTED;
  cudaError_t e = cudaMemsetAsync(p.flags, 0, lay.flag_bytes, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  int rc = trace_mark(g_trace_begin, stream);
  if (rc != DILATTN_OK) return rc;
  if (units > 0)
    fwd_tile_kernel<D, QK8>
        <<<(unsigned)units, FwdCfg<D, QK8>::THREADS, FwdCfg<D, QK8>::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "fwd_tile_kernel launch");
  rc = trace_mark(g_trace_end, stream);
  if (rc != DILATTN_OK) return rc;
  if (p.merger >= 0) return DILATTN_OK;

  // No pattern keeps every row: a separate pass merges the partials.
  MergeParams mp;
  memset(&mp, 0, sizeof(mp));
  memcpy(mp.pat, p.pat, sizeof(mp.pat));
  mp.npat = npat;
  mp.B = B;
  mp.N = N;
  mp.H = H;
  mp.part_o = p.part_o;
  mp.part_lse = p.part_lse;
  mp.out = reinterpret_cast<__nv_bfloat16*>(out);
  mp.out_res = reinterpret_cast<__nv_bfloat16*>(out_res);
  mp.lse = lse;
  const long long total_rows = (long long)B * N * H;
  constexpr int rows_per_block = 256 / kMergeTpr;
  const long long blocks = (total_rows + rows_per_block - 1) / rows_per_block;
  merge_kernel<D><<<(unsigned)blocks, 256, 0, stream>>>(mp);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "merge_kernel launch");
  return DILATTN_OK;
}

int launch_bwd(const void* q, const void* k, const void* v, const void* out, const void* out_res,
               const float* lse, const void* dout, float* dq, float* dk, float* dv, int B, int N,
               int H,
               const int* w, const int* r, int npat, int causal, void* ws,
               DeviceState* st, cudaStream_t stream) {
  NvtxRange range("dilattn backward");
  constexpr int D = 64;
  static_assert(sizeof(BwdParams) < 32000, "kernel parameter block too large");
  BwdParams p;
  memset(&p, 0, sizeof(p));
  p.npat = npat;
  p.B = B;
  p.N = N;
  p.H = H;
  p.causal = causal;
  p.tau = (float)(1.0 / std::sqrt((double)D));
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D));
  make_geoms(B, N, H, w, r, npat, p.pat);
  // workspace: D [B][H][N] fp32, 256 bytes for the key-tile kernel's unit
  // counter, then fp16 copies of q and k
  char* wsb = reinterpret_cast<char*>(ws);
  float* drow = reinterpret_cast<float*>(wsb);
  p.drow = drow;
  p.lse = lse;
  const size_t dbytes = align256((size_t)B * H * N * 4);
  p.counter = reinterpret_cast<int*>(wsb + dbytes);
  __half* q16 = reinterpret_cast<__half*>(wsb + dbytes + 256);
  __half* k16 = reinterpret_cast<__half*>(wsb + dbytes + 256 + align256((size_t)B * N * H * D * 2));
  p.err = ErrCtx{st->err_word, next_tag()};
  for (int i = 0; i < npat; ++i) {
    const void* src[4] = {q16, k16, v, dout};
    const int dtype[4] = {2, 2, 0, 0};
    CUtensorMap* dst[4] = {&p.tmq[i], &p.tmk[i], &p.tmv[i], &p.tmdo[i]};
    CUtensorMap* dst_t[4] = {&p.tmq_t[i], &p.tmk_t[i], &p.tmv_t[i], &p.tmdo_t[i]};
    for (int j = 0; j < 4; ++j) {
      int rc = strided_map(src[j], B, N, H, D, r[i], 0, dst[j], dtype[j]);
      if (rc == DILATTN_OK) rc = strided_map(src[j], B, N, H, D, r[i], 1, dst_t[j], dtype[j]);
      if (rc != DILATTN_OK) return rc;
    }
    // reduce-add targets: one row warp adds a 32-row x 32-column block
    const float* grad[3] = {dq, dk, dv};
    CUtensorMap* gm[3] = {&p.tmdq[i], &p.tmdk[i], &p.tmdv[i]};
    CUtensorMap* gm_t[3] = {&p.tmdq_t[i], &p.tmdk_t[i], &p.tmdv_t[i]};
    for (int j = 0; j < 3; ++j) {
      int rc = strided_map(grad[j], B, N, H, D, r[i], 0, gm[j], 1, 32);
      if (rc == DILATTN_OK) rc = strided_map(grad[j], B, N, H, D, r[i], 1, gm_t[j], 1, 32);
      if (rc != DILATTN_OK) return rc;
    }
  }
  // group-major unit order: patterns by tile count (descending, stable), then
  // (segment, batch, head) groups, then key tiles
  {
    std::vector<int> order(npat);
    for (int i = 0; i < npat; ++i) order[i] = i;
    std::stable_sort(order.begin(), order.end(),
                     [&](int a, int b) { return p.pat[a].ntiles > p.pat[b].ntiles; });
    p.gstart[0] = 0;
    for (int a = 0; a < npat; ++a) {
      const PatternGeom& g = p.pat[order[a]];
      p.gorder[a] = order[a];
      p.gstart[a + 1] = p.gstart[a] + (long long)g.nseg * B * H * g.ntiles;
    }
  }
  const long long units = p.gstart[npat];
  if (units > 0x7fffffffLL) return DILATTN_ERR_UNSUPPORTED;
  const long long rows = (long long)B * N * H;

  PrepParams pp;
  pp.B = B;
  pp.N = N;
  pp.H = H;
  pp.q = reinterpret_cast<const __nv_bfloat16*>(q);
  pp.k = reinterpret_cast<const __nv_bfloat16*>(k);
  pp.q16 = q16;
  pp.k16 = k16;
  pp.err = p.err;
  pp.out = reinterpret_cast<const __nv_bfloat16*>(out);
  pp.out_res = reinterpret_cast<const __nv_bfloat16*>(out_res);
  pp.dout = reinterpret_cast<const __nv_bfloat16*>(dout);
  pp.drow = drow;
  pp.dq = dq;
  pp.dk = dk;
  pp.dv = dv;
  pp.counter = p.counter;
  bwd_prep_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, stream>>>(pp);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "bwd_prep_kernel launch");
  int rc = trace_mark(g_trace_begin, stream);
  if (rc != DILATTN_OK) return rc;
  // persistent: one CTA per SM, each taking units of the longest-first list from the counter
  p.units = units;
  const long long grid = std::min<long long>(units, (long long)st->num_sms);
  if (grid > 0)
    bwd_tile_kernel<<<(unsigned)grid, BwdCfg::THREADS, BwdCfg::SMEM_BYTES, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "bwd_tile_kernel launch");
  return trace_mark(g_trace_end, stream);
}

RowParams make_row_params(int B, int N, int H, int d, const int* w, const int* r, int npat,
                          int causal) {
  RowParams p;
  memset(&p, 0, sizeof(p));
  make_geoms(B, N, H, w, r, npat, p.pat);
  p.npat = npat;
  p.B = B;
  p.N = N;
  p.H = H;
  p.causal = causal;
  p.tau = (float)(1.0 / std::sqrt((double)d));
  return p;
}

}  // namespace
}  // namespace dil

using namespace dil;

extern "C" {

const char* dilattn_status_string(int status) {
  switch (status) {
    case DILATTN_OK: return "DILATTN_OK";
    case DILATTN_ERR_INVALID_ARG: return "DILATTN_ERR_INVALID_ARG";
    case DILATTN_ERR_UNSUPPORTED: return "DILATTN_ERR_UNSUPPORTED";
    case DILATTN_ERR_CUDA: return "DILATTN_ERR_CUDA";
    case DILATTN_ERR_WORKSPACE: return "DILATTN_ERR_WORKSPACE";
    case DILATTN_ERR_INTERNAL: return "DILATTN_ERR_INTERNAL";
    default: return "DILATTN_UNKNOWN_STATUS";
  }
}

const char* dilattn_last_error(void) { return g_last_error; }

size_t dilattn_fwd_scratch_size(int B, int N, int H, int d, const int* w, const int* r,
                                int npat) {
  if (check_shape(B, N, H, d, w, r, npat, 1) != DILATTN_OK) return 0;
  return fwd_scratch_bytes(B, N, H, d, w, r, npat);
}

}  // extern "C"

namespace dil {
namespace {
// dilattn_fwd and dilattn_fwd_train: scratch from the library's pool.
int fwd_pooled(const void* q, const void* k, const void* v, void* out, void* out_res, float* lse,
               int B, int N, int H, int d, const int* w, const int* r, int npat, int causal,
               cudaStream_t stream) {
  int rc = check_fwd_args(q, k, v, out, lse, B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  if (out_res != nullptr) {
    const size_t tb = (size_t)B * N * H * d * 2;
    if (!aligned16(out_res) || overlaps(out_res, tb, q, tb) || overlaps(out_res, tb, k, tb) ||
        overlaps(out_res, tb, v, tb) || overlaps(out_res, tb, out, tb) ||
        (lse != nullptr && overlaps(out_res, tb, lse, (size_t)B * H * N * 4)))
      return DILATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  cudaMemPool_t pool = nullptr;
  rc = scratch_pool(st, &pool);
  if (rc != DILATTN_OK) return rc;
  const size_t need = fwd_scratch_bytes(B, N, H, d, w, r, npat);
  void* scratch = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&scratch, need, pool, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync (forward scratch)");
  rc = d == 64 ? launch_fwd<64>(q, k, v, out, out_res, lse, B, N, H, w, r, npat, causal, scratch,
                                st, stream)
               : launch_fwd<128>(q, k, v, out, out_res, lse, B, N, H, w, r, npat, causal, scratch,
                                 st, stream);
  e = cudaFreeAsync(scratch, stream);  // stream-ordered: after the kernels that use it
  if (rc == DILATTN_OK && e != cudaSuccess) return cuda_fail(e, "cudaFreeAsync (forward scratch)");
  return rc;
}
}  // namespace
}  // namespace dil

extern "C" {

int dilattn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int N,
                int H, int d, const int* w, const int* r, int npat, int causal,
                cudaStream_t stream) {
  return fwd_pooled(q, k, v, out, nullptr, lse, B, N, H, d, w, r, npat, causal, stream);
}

int dilattn_fwd_fp8(const void* q8, const void* k8, const void* v, void* out, float* lse, int B,
                    int N, int H, int d, const int* w, const int* r, int npat, int causal,
                    float q_scale, float k_scale, cudaStream_t stream) {
  int rc = check_shape(B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  if (d != 128) {
    snprintf(g_last_error, sizeof(g_last_error), "the fp8 forward is built for d = 128");
    return DILATTN_ERR_UNSUPPORTED;
  }
  if (!(q_scale > 0.f) || !(k_scale > 0.f) || !std::isfinite(q_scale) || !std::isfinite(k_scale))
    return DILATTN_ERR_INVALID_ARG;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(v) || !aligned16(out) ||
      (lse != nullptr && !aligned16(lse)))
    return DILATTN_ERR_INVALID_ARG;
  const size_t t8 = (size_t)B * N * H * d, tb = 2 * t8, lb = (size_t)B * H * N * 4;
  if (overlaps(out, tb, q8, t8) || overlaps(out, tb, k8, t8) || overlaps(out, tb, v, tb) ||
      (lse != nullptr && (overlaps(lse, lb, q8, t8) || overlaps(lse, lb, k8, t8) ||
                          overlaps(lse, lb, v, tb) || overlaps(lse, lb, out, tb))))
    return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  cudaMemPool_t pool = nullptr;
  rc = scratch_pool(st, &pool);
  if (rc != DILATTN_OK) return rc;
  const size_t need = fwd_scratch_bytes(B, N, H, d, w, r, npat);
  void* scratch = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&scratch, need, pool, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync (forward scratch)");
  rc = launch_fwd<128, true>(q8, k8, v, out, nullptr, lse, B, N, H, w, r, npat, causal, scratch,
                             st, stream, nullptr, q_scale * k_scale);
  e = cudaFreeAsync(scratch, stream);
  if (rc == DILATTN_OK && e != cudaSuccess) return cuda_fail(e, "cudaFreeAsync (forward scratch)");
  return rc;
}

int dilattn_fwd_train(const void* q, const void* k, const void* v, void* out, void* out_res,
                      float* lse, int B, int N, int H, int d, const int* w, const int* r, int npat,
                      int causal, cudaStream_t stream) {
  if (out_res == nullptr) return DILATTN_ERR_INVALID_ARG;
  return fwd_pooled(q, k, v, out, out_res, lse, B, N, H, d, w, r, npat, causal, stream);
}

size_t dilattn_bwd_workspace_size(int B, int N, int H, int d) {
  if (B < 1 || N < 1 || H < 1 || d < 1 || (double)B * N * H * d >= 1099511627776.0) return 0;
  // D, the unit counter, then fp16 copies of q and k
  return align256((size_t)B * H * N * 4) + 256 + 2 * align256((size_t)B * N * H * d * 2);
}

int dilattn_bwd(const void* q, const void* k, const void* v, const void* out,
                const void* out_res, const float* lse, const void* dout, float* dq, float* dk,
                float* dv, int B, int N, int H, int d, const int* w, const int* r, int npat,
                int causal, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_shape(B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  const void* ins[7] = {q, k, v, out, lse, dout, out_res};
  for (const void* x : ins)
    if (!aligned16(x)) return DILATTN_ERR_INVALID_ARG;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return DILATTN_ERR_INVALID_ARG;
  const size_t tb = (size_t)B * N * H * d * 2;  // a bf16 input
  const size_t gb = 2 * tb;                     // an fp32 gradient
  const size_t lb = (size_t)B * H * N * 4;
  void* outs[3] = {dq, dk, dv};
  for (void* o : outs)
    for (int j = 0; j < 7; ++j)
      if (overlaps(o, gb, ins[j], j == 4 ? lb : tb)) return DILATTN_ERR_INVALID_ARG;
  if (overlaps(dq, gb, dk, gb) || overlaps(dq, gb, dv, gb) || overlaps(dk, gb, dv, gb))
    return DILATTN_ERR_INVALID_ARG;
  if (d != 64) {
    snprintf(g_last_error, sizeof(g_last_error), "bf16 backward is built for d = 64");
    return DILATTN_ERR_UNSUPPORTED;
  }
  const size_t need = dilattn_bwd_workspace_size(B, N, H, d);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 ||
      workspace_bytes < need)
    return DILATTN_ERR_WORKSPACE;
  for (int j = 0; j < 7; ++j)
    if (overlaps(workspace, need, ins[j], j == 4 ? lb : tb)) return DILATTN_ERR_INVALID_ARG;
  for (void* o : outs)
    if (overlaps(workspace, need, o, gb)) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  return launch_bwd(q, k, v, out, out_res, lse, dout, dq, dk, dv, B, N, H, w, r, npat, causal,
                    workspace, st, stream);
}

int dilattn_fwd_f32(const float* q, const float* k, const float* v, float* out, float* lse, int B,
                    int N, int H, int d, const int* w, const int* r, int npat, int causal,
                    cudaStream_t stream) {
  int rc = check_shape(B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return DILATTN_ERR_INVALID_ARG;
  if (lse != nullptr && !aligned16(lse)) return DILATTN_ERR_INVALID_ARG;
  const size_t tb = (size_t)B * N * H * d * 4;
  if (overlaps(out, tb, q, tb) || overlaps(out, tb, k, tb) || overlaps(out, tb, v, tb))
    return DILATTN_ERR_INVALID_ARG;
  if (lse != nullptr) {
    const size_t lb = (size_t)B * H * N * 4;
    if (overlaps(lse, lb, q, tb) || overlaps(lse, lb, k, tb) || overlaps(lse, lb, v, tb) ||
        overlaps(lse, lb, out, tb))
      return DILATTN_ERR_INVALID_ARG;
  }
  if (d != 64 && d != 128) return DILATTN_ERR_UNSUPPORTED;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  RowParams p = make_row_params(B, N, H, d, w, r, npat, causal);
  const long long rows = (long long)B * N * H;
  const unsigned blocks = (unsigned)((rows + 127) / 128);
  if (d == 64)
    fwd_f32_kernel<64><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse);
  else
    fwd_f32_kernel<128><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "fwd_f32_kernel launch");
  return DILATTN_OK;
}

int dilattn_bwd_f32(const float* q, const float* k, const float* v, const float* out,
                    const float* lse, const float* dout, float* dq, float* dk, float* dv, int B,
                    int N, int H, int d, const int* w, const int* r, int npat, int causal,
                    cudaStream_t stream) {
  int rc = check_shape(B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  const void* ins[6] = {q, k, v, out, lse, dout};
  for (const void* x : ins)
    if (!aligned16(x)) return DILATTN_ERR_INVALID_ARG;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv)) return DILATTN_ERR_INVALID_ARG;
  const size_t tb = (size_t)B * N * H * d * 4;
  const size_t lb = (size_t)B * H * N * 4;
  void* outs[3] = {dq, dk, dv};
  for (void* o : outs) {
    for (int j = 0; j < 6; ++j)
      if (overlaps(o, tb, ins[j], j == 4 ? lb : tb)) return DILATTN_ERR_INVALID_ARG;
  }
  if (overlaps(dq, tb, dk, tb) || overlaps(dq, tb, dv, tb) || overlaps(dk, tb, dv, tb))
    return DILATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return DILATTN_ERR_UNSUPPORTED;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  RowParams p = make_row_params(B, N, H, d, w, r, npat, causal);
  const long long rows = (long long)B * N * H;
  const unsigned blocks = (unsigned)((rows + 127) / 128);
  if (d == 64) {
    bwd_dq_f32_kernel<64><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse, dout, dq);
    bwd_dkdv_f32_kernel<64><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse, dout, dk, dv);
  } else {
    bwd_dq_f32_kernel<128><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse, dout, dq);
    bwd_dkdv_f32_kernel<128><<<blocks, 128, 0, stream>>>(p, q, k, v, out, lse, dout, dk, dv);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "bwd_f32 launch");
  return DILATTN_OK;
}

int dilattn_selection(uint32_t* sig, int N, int H, const int* w, const int* r, int npat,
                      cudaStream_t stream) {
  int rc = check_shape(1, N, H, 1, w, r, npat, 1);
  if (rc != DILATTN_OK) return rc;
  if (!aligned16(sig)) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  PatternGeom geo[kMaxPat];
  make_geoms(1, N, H, w, r, npat, geo);
  cudaError_t e = cudaMemsetAsync(sig, 0, (size_t)H * N * 4, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
  for (int i = 0; i < npat; ++i) {
    const long long gx = (long long)geo[i].nseg * H;
    if (gx > 0x7fffffffLL) return DILATTN_ERR_UNSUPPORTED;
    const int gy = std::min(64, (geo[i].nmax + 255) / 256);
    selection_kernel<<<dim3((unsigned)gx, gy), 256, 0, stream>>>(geo[i], i, N, H, sig);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "selection_kernel launch");
  return DILATTN_OK;
}

int dilattn_pack_dilated(const void* x, void* buf, int B, int L, int H, int d, int r,
                         cudaStream_t stream) {
  if (B < 1 || L < 1 || H < 1 || r < 1 || L % r != 0 || (d != 64 && d != 128))
    return DILATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(buf)) return DILATTN_ERR_INVALID_ARG;
  const size_t bytes = (size_t)B * L * H * d * 2;
  if (overlaps(x, bytes, buf, bytes / r)) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  const long long n16 = (long long)B * (L / r) * H * (d / 8);  // 16-byte pieces
  const long long blocks = std::min<long long>((n16 + 255) / 256, (long long)st->num_sms * 32);
  pack_dilated_kernel<<<(unsigned)blocks, 256, 0, stream>>>(
      reinterpret_cast<const uint4*>(x), reinterpret_cast<uint4*>(buf), B, L, H, d / 8, r);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "pack_dilated_kernel launch");
  return DILATTN_OK;
}

int dilattn_fwd_seqpar(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                       int L, int H, int d, const int* w, const int* r, int npat, int causal,
                       int rank, int world, const void* const* kg, const void* const* vg,
                       cudaStream_t stream) {
  int rc = check_fwd_args(q, k, v, out, lse, B, L, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  if (world < 1 || rank < 0 || rank >= world || (long long)L * world > 0x7fffffffLL)
    return DILATTN_ERR_INVALID_ARG;
  const long long N = (long long)L * world;
  SeqParPlan sp;
  memset(&sp, 0, sizeof(sp));
  int wl[kMaxPat];
  for (int i = 0; i < npat; ++i) {
    if (w[i] <= L) {  // every segment lies in one rank's block
      if (L % w[i] != 0) return DILATTN_ERR_INVALID_ARG;
      wl[i] = w[i];
      continue;
    }
    const long long span = std::min<long long>(w[i], N);  // a segment spans span / L ranks
    if (span % L != 0 || (w[i] < N && N % w[i] != 0) || L % r[i] != 0 || (L / r[i]) % BM != 0)
      return DILATTN_ERR_INVALID_ARG;
    if (kg == nullptr || vg == nullptr || !aligned16(kg[i]) || !aligned16(vg[i]))
      return DILATTN_ERR_INVALID_ARG;
    wl[i] = L;  // this rank's kept rows: offset h mod r, stride r, over its whole block
    sp.ranks[i] = (int)(span / L);
    sp.kv_rank_rows[i] = L / r[i];
    sp.kv_rows[i] = sp.ranks[i] * sp.kv_rank_rows[i];
    sp.toff[i] = (rank % sp.ranks[i]) * (sp.kv_rank_rows[i] / BM);
    sp.kg[i] = kg[i];
    sp.vg[i] = vg[i];
    // the gathered rows are read while out and lse are written
    const size_t gb = (size_t)sp.kv_rows[i] * B * H * d * 2;
    const size_t tb = (size_t)B * L * H * d * 2, lb = (size_t)B * H * L * 4;
    if (overlaps(out, tb, kg[i], gb) || overlaps(out, tb, vg[i], gb) ||
        (lse != nullptr && (overlaps(lse, lb, kg[i], gb) || overlaps(lse, lb, vg[i], gb))))
      return DILATTN_ERR_INVALID_ARG;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  cudaMemPool_t pool = nullptr;
  rc = scratch_pool(st, &pool);
  if (rc != DILATTN_OK) return rc;
  const size_t need = fwd_scratch_bytes(B, L, H, d, wl, r, npat);
  void* scratch = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&scratch, need, pool, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync (forward scratch)");
  rc = d == 64
      ? launch_fwd<64>(q, k, v, out, nullptr, lse, B, L, H, wl, r, npat, causal, scratch, st,
                       stream, &sp)
      : launch_fwd<128>(q, k, v, out, nullptr, lse, B, L, H, wl, r, npat, causal, scratch, st,
                        stream, &sp);
  e = cudaFreeAsync(scratch, stream);
  if (rc == DILATTN_OK && e != cudaSuccess) return cuda_fail(e, "cudaFreeAsync (forward scratch)");
  return rc;
}

int dilattn_set_trace_events(cudaEvent_t tile_begin, cudaEvent_t tile_end) {
  if ((tile_begin == nullptr) != (tile_end == nullptr)) return DILATTN_ERR_INVALID_ARG;
  g_trace_begin = tile_begin;
  g_trace_end = tile_end;
  return DILATTN_OK;
}

int dilattn_device_error(cudaStream_t stream, int* code) {
  if (code == nullptr) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int v = 0;
  e = cudaMemcpy(&v, st->err_word, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy");
  const int zero = 0;
  e = cudaMemcpy(st->err_word, &zero, sizeof(int), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpy");
  *code = v & 0xff;  // the word holds (launch tag << 8) | code
  return DILATTN_OK;
}

int dilattn_selftest_wait_timeout(unsigned long long limit_ns, int* result, cudaStream_t stream) {
  if (result == nullptr || !aligned16(result) || limit_ns == 0 || limit_ns > 1000000000ull)
    return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  int rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  selftest_wait_kernel<<<1, 64, 0, stream>>>(ErrCtx{st->err_word, next_tag()}, limit_ns, result);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "selftest_wait_kernel launch");
  return DILATTN_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Forward with a scratch array compiled into the library (no allocation)
// ---------------------------------------------------------------------------
namespace dil {

// Scratch of dilattn_fwd_noalloc. In host code this name is only a stand-in
// for the device array: kernels get the address cudaGetSymbolAddress returns.
static __device__ __align__(256) unsigned char g_noalloc_scratch[DILATTN_NOALLOC_SCRATCH_BYTES];

namespace {
std::mutex g_noalloc_mu;
std::map<int, void*> g_noalloc_addr;  // device ordinal -> device address of the scratch

// Device address of the scratch on the current device, looked up once per device.
int noalloc_scratch(void** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  auto it = g_noalloc_addr.find(dev);
  if (it == g_noalloc_addr.end()) {
    void* ptr = nullptr;
    e = cudaGetSymbolAddress(&ptr, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(g_noalloc_scratch)");
    it = g_noalloc_addr.emplace(dev, ptr).first;
  }
  *out = it->second;
  return DILATTN_OK;
}
}  // namespace
}  // namespace dil

extern "C" int dilattn_fwd_noalloc(const void* q, const void* k, const void* v, void* out,
                                   float* lse, int B, int N, int H, int d, const int* w,
                                   const int* r, int npat, int causal, cudaStream_t stream) {
  int rc = check_fwd_args(q, k, v, out, lse, B, N, H, d, w, r, npat, causal);
  if (rc != DILATTN_OK) return rc;
  const size_t need = fwd_scratch_bytes(B, N, H, d, w, r, npat);
  if (need > (size_t)DILATTN_NOALLOC_SCRATCH_BYTES) {
    snprintf(g_last_error, sizeof(g_last_error),
             "dilattn_fwd_noalloc: this problem needs %zu bytes of scratch; the built-in "
             "scratch holds %zu bytes (use dilattn_fwd)",
             need, (size_t)DILATTN_NOALLOC_SCRATCH_BYTES);
    return DILATTN_ERR_WORKSPACE;
  }
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  void* scratch = nullptr;
  rc = noalloc_scratch(&scratch);
  if (rc != DILATTN_OK) return rc;
  if (d == 64)
    return launch_fwd<64>(q, k, v, out, nullptr, lse, B, N, H, w, r, npat, causal, scratch, st,
                          stream);
  return launch_fwd<128>(q, k, v, out, nullptr, lse, B, N, H, w, r, npat, causal, scratch, st,
                         stream);
}

// ---------------------------------------------------------------------------
// The 8-bit key/value cache and the attention over it
// ---------------------------------------------------------------------------
namespace dil {
namespace {

// A buffer as the overlap checks see it.
struct Span {
  const void* p;
  size_t n;
};

// The checks that every cache entry point makes of the cache and its table.
int check_cache(const void* kc, const void* vc, const float* ks, const float* vs, int pages,
                int Hkv, int page_size, int d, int format, const int* table, int B,
                int max_pages) {
  if (pages < 1 || Hkv < 1 || B < 1 || max_pages < 1) return DILATTN_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return DILATTN_ERR_INVALID_ARG;
  if (format != DILATTN_CACHE_E4M3 && format != DILATTN_CACHE_INT8) return DILATTN_ERR_INVALID_ARG;
  // cache rows are counted in 32 bits, positions in 31, the sequences of a warp's search in 30
  if (B >= (1 << 30) || (double)pages * Hkv * page_size >= 4294967295.0 ||
      (double)max_pages * page_size > 2147483647.0)
    return DILATTN_ERR_INVALID_ARG;
  if (!aligned16(kc) || !aligned16(vc) || !aligned16(ks) || !aligned16(vs) || !aligned4(table))
    return DILATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return DILATTN_ERR_UNSUPPORTED;
  const size_t cb = (size_t)pages * Hkv * page_size * d, sb = (size_t)pages * Hkv * 4;
  const Span s[5] = {{kc, cb}, {vc, cb}, {ks, sb}, {vs, sb}, {table, (size_t)B * max_pages * 4}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(s[i].p, s[i].n, s[j].p, s[j].n)) return DILATTN_ERR_INVALID_ARG;
  return DILATTN_OK;
}

// Bytes from the first element to the last of n rows of `row` 2-byte elements, `stride` apart.
size_t strided_bytes(long long n, long long row, long long stride) {
  return n < 1 ? 0 : (size_t)((n - 1) * stride + row) * 2;
}

// Whether two sets of n rows of `row` 2-byte elements share an element. Sets
// of the same stride may interleave, as slices of one buffer do: then their
// rows are `shift` bytes apart, modulo the stride.
bool rows_overlap(const void* a, long long a_stride, const void* b, long long b_stride,
                  long long n, long long row) {
  if (!overlaps(a, strided_bytes(n, row, a_stride), b, strided_bytes(n, row, b_stride)))
    return false;
  if (a_stride != b_stride) return true;
  const long long shift = std::llabs((const char*)a - (const char*)b) % (2 * a_stride);
  return shift < 2 * row || shift > 2 * (a_stride - row);
}

// Row strides count elements: at least one row, and 16-byte aligned.
bool good_stride(long long stride, long long row) {
  return stride >= row && stride % 8 == 0 && stride < (1ll << 40);
}

CacheGeom cache_geom(const int* table, int B, int max_pages, int pages, int Hkv, int page_size,
                     DeviceState* st) {
  CacheGeom g;
  g.table = table;
  g.B = B;
  g.max_pages = max_pages;
  g.pages = pages;
  g.Hkv = Hkv;
  g.lp = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  g.err = ErrCtx{st->err_word, next_tag()};
  return g;
}

// Checks of the ragged token batch that writes and reads share.
int check_tokens(const void* k, const void* v, long long k_stride, long long v_stride,
                 const int* offsets, const int* start, int T, int B, int Hkv, int d) {
  if (T < 0 || (offsets == nullptr && T != B)) return DILATTN_ERR_INVALID_ARG;
  if (!aligned4(start) || (offsets != nullptr && !aligned4(offsets)))
    return DILATTN_ERR_INVALID_ARG;
  const long long row = (long long)Hkv * d;
  if (T > 0 && (!aligned16(k) || !aligned16(v))) return DILATTN_ERR_INVALID_ARG;
  if (!good_stride(k_stride, row) || !good_stride(v_stride, row)) return DILATTN_ERR_INVALID_ARG;
  return DILATTN_OK;
}

// A launch that may start while the kernel before it on the stream still
// runs; the kernel itself waits for that one's end before it reads its results.
template <typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Args...), dim3 grid, int threads, size_t smem,
                              cudaStream_t stream, int cluster, Args... args) {
  cudaLaunchAttribute attr[2];
  memset(attr, 0, sizeof(attr));
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int FMT>
cudaError_t launch_cache_write(const CacheWriteParams& p, long long slots, int page_size, cudaStream_t stream) {
  const long long units = slots * p.geom.Hkv;
  // few tokens of each sequence (on average, which is all that the host knows): a warp a page, which
  // does not idle where a page has few new rows. At 1, 8 and 16 tokens of each of 64 sequences of 32 heads it takes 5, 7 and 10 us where the other
  // takes 23, 25 and 27, of 16 sequences of 12 heads 2.7, 3.2 and 4.1 against 3.9, 3.9 and 4.0
  if (p.tok.offsets == nullptr || p.tok.T <= 8 * (long long)p.geom.B)
    return launch_overlapped(cache_append_kernel<D, FMT>, dim3((unsigned)((2 * units + 7) / 8)), 256, 0, stream, 1,
                             p);
  // 64 numbers a lane, 32 where a page and head has no more for a warp (33 against 45 us for 29
  // ragged prompts over 16-token pages, d = 64; elsewhere 32 are up to 4% slower)
  const int size = page_size * D, warps = std::max(1, size / 2048);
  const dim3 grid((unsigned)((units * warps + 7) / 8));
  const auto kernel = size == 1024 ? cache_write_kernel<D, FMT, 1, D / 32>
                      : warps == 1 ? cache_write_kernel<D, FMT, 1, 4>
                      : warps == 2 ? cache_write_kernel<D, FMT, 2, 4>
                      : warps == 4 ? cache_write_kernel<D, FMT, 4, 4>
                                   : cache_write_kernel<D, FMT, D / 16, 4>;
  return launch_overlapped(kernel, grid, 256, 0, stream, 1, p);
}

template <int D, int FMT>
cudaError_t launch_cache_read(const CacheReadParams& p, int num_sms, cudaStream_t stream) {
  // one piece a thread while every thread runs at once (3 against 3.6 us for a few tokens), then
  // two, whose loads overlap (506 against 590 us for 131072 tokens of 32 heads, d = 128)
  const long long all = (long long)p.tok.T * p.pieces;
  const int each = all <= 2048ll * num_sms ? 1 : 2;
  const dim3 grid((unsigned)((all + kReadThreads * each - 1) / (kReadThreads * each)), 2);
  const auto kernel = each == 1 ? cache_read_kernel<D, FMT, 1> : cache_read_kernel<D, FMT, 2>;
  return launch_overlapped(kernel, grid, kReadThreads, 0, stream, 1, p);
}

// Whether a written buffer overlaps a read one.
bool any_overlap(const Span* mut, int nm, const Span* ro, int nr) {
  for (int i = 0; i < nm; ++i)
    for (int j = 0; j < nr; ++j)
      if (overlaps(mut[i].p, mut[i].n, ro[j].p, ro[j].n)) return true;
  return false;
}

}  // namespace
}  // namespace dil

extern "C" int dilattn_cache_write(const void* k, const void* v, long long k_stride,
                                   long long v_stride, const int* offsets, const int* start,
                                   int T, const int* table, int B, int max_pages, void* kc,
                                   void* vc, float* ks, float* vs, int pages, int Hkv,
                                   int page_size, int d, int format, cudaStream_t stream) {
  int rc = check_cache(kc, vc, ks, vs, pages, Hkv, page_size, d, format, table, B, max_pages);
  if (rc != DILATTN_OK) return rc;
  rc = check_tokens(k, v, k_stride, v_stride, offsets, start, T, B, Hkv, d);
  if (rc != DILATTN_OK) return rc;
  if (T == 0) return DILATTN_OK;
  const size_t cb = (size_t)pages * Hkv * page_size * d, sb = (size_t)pages * Hkv * 4;
  const long long row = (long long)Hkv * d;
  const Span mut[4] = {{kc, cb}, {vc, cb}, {ks, sb}, {vs, sb}};
  const Span ro[4] = {{k, strided_bytes(T, row, k_stride)},
                      {v, strided_bytes(T, row, v_stride)},
                      {start, (size_t)B * 4},
                      {offsets, offsets != nullptr ? (size_t)(B + 1) * 4 : 0}};
  if (any_overlap(mut, 4, ro, 4)) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  NvtxRange range("dilattn cache write");
  CacheWriteParams p;
  p.geom = cache_geom(table, B, max_pages, pages, Hkv, page_size, st);
  p.tok = CacheTokens{offsets, start, T};
  p.x[0] = reinterpret_cast<const __nv_bfloat16*>(k);
  p.x[1] = reinterpret_cast<const __nv_bfloat16*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.codes[0] = reinterpret_cast<uint8_t*>(kc);
  p.codes[1] = reinterpret_cast<uint8_t*>(vc);
  p.scale[0] = ks;
  p.scale[1] = vs;
  const long long slots = offsets == nullptr ? B : (long long)T / page_size + 2ll * B + 1;
  if ((double)slots * Hkv * 8 > 2147483647.0) return DILATTN_ERR_UNSUPPORTED;
  divisor_magic((uint32_t)Hkv, p.h_mul, p.h_sh);
  cudaError_t e;
  if (format == DILATTN_CACHE_E4M3)
    e = d == 64 ? launch_cache_write<64, kFmtE4M3>(p, slots, page_size, stream)
                : launch_cache_write<128, kFmtE4M3>(p, slots, page_size, stream);
  else
    e = d == 64 ? launch_cache_write<64, kFmtInt8>(p, slots, page_size, stream)
                : launch_cache_write<128, kFmtInt8>(p, slots, page_size, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache write launch");
  return DILATTN_OK;
}

extern "C" int dilattn_cache_read(const void* kc, const void* vc, const float* ks,
                                  const float* vs, int pages, int Hkv, int page_size, int d,
                                  int format, const int* table, int B, int max_pages,
                                  const int* offsets, const int* start, int T, void* k, void* v,
                                  long long k_stride, long long v_stride, cudaStream_t stream) {
  int rc = check_cache(kc, vc, ks, vs, pages, Hkv, page_size, d, format, table, B, max_pages);
  if (rc != DILATTN_OK) return rc;
  rc = check_tokens(k, v, k_stride, v_stride, offsets, start, T, B, Hkv, d);
  if (rc != DILATTN_OK) return rc;
  if (T == 0) return DILATTN_OK;
  const size_t cb = (size_t)pages * Hkv * page_size * d, sb = (size_t)pages * Hkv * 4;
  const long long row = (long long)Hkv * d;
  if (rows_overlap(k, k_stride, v, v_stride, T, row)) return DILATTN_ERR_INVALID_ARG;
  const Span mut[2] = {{k, strided_bytes(T, row, k_stride)}, {v, strided_bytes(T, row, v_stride)}};
  const Span ro[7] = {{kc, cb}, {vc, cb}, {ks, sb}, {vs, sb},
                      {table, (size_t)B * max_pages * 4}, {start, (size_t)B * 4},
                      {offsets, offsets != nullptr ? (size_t)(B + 1) * 4 : 0}};
  if (any_overlap(mut, 2, ro, 7)) return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  NvtxRange range("dilattn cache read");
  CacheReadParams p;
  p.geom = cache_geom(table, B, max_pages, pages, Hkv, page_size, st);
  p.tok = CacheTokens{offsets, start, T};
  p.x[0] = reinterpret_cast<__nv_bfloat16*>(k);
  p.x[1] = reinterpret_cast<__nv_bfloat16*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.codes[0] = reinterpret_cast<const uint8_t*>(kc);
  p.codes[1] = reinterpret_cast<const uint8_t*>(vc);
  p.scale[0] = ks;
  p.scale[1] = vs;
  const long long most = (long long)Hkv * (d / 16);
  if (most > 0x3fffffffLL || (double)T * most / kReadThreads > 2147483647.0) return DILATTN_ERR_UNSUPPORTED;
  p.pieces = (int)most;
  divisor_magic((uint32_t)p.pieces, p.p_mul, p.p_sh);
  cudaError_t e;
  if (format == DILATTN_CACHE_E4M3)
    e = d == 64 ? launch_cache_read<64, kFmtE4M3>(p, st->num_sms, stream)
                : launch_cache_read<128, kFmtE4M3>(p, st->num_sms, stream);
  else
    e = d == 64 ? launch_cache_read<64, kFmtInt8>(p, st->num_sms, stream)
                : launch_cache_read<128, kFmtInt8>(p, st->num_sms, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache_read_kernel launch");
  return DILATTN_OK;
}

namespace dil {
namespace {

// Columns of an item: a power of two up to 8, or 16; what a decode kernel is made for. `grouped`:
// its columns are the heads of several tokens.
int decode_heads(int G, bool grouped) {
  if (grouped) return G <= 4 ? 8 : 16;
  return G <= 2 ? G : G <= 4 ? 4 : G <= 8 ? 8 : 16;
}
int decode_tokens(int G, bool grouped) { return grouped ? decode_heads(G, true) / G : 1; }
int decode_columns(int G, bool grouped) { return std::min(G * decode_tokens(G, grouped), decode_heads(G, grouped)); }
long long decode_items(int T, int Hkv, int G, bool grouped) {
  const int heads = decode_heads(G, grouped), tokens = decode_tokens(G, grouped);
  return ((long long)T + tokens - 1) / tokens * Hkv * (grouped ? 1 : (G + heads - 1) / heads);
}

// Blocks of a team for `items` items of up to `tiles` tiles (see decode_team_kernel), or -1: they
// are too many or too long, and ranges of all items' tiles serve better. Up to eight tiles are
// done by a warp before more of them would have met. Teams of blocks all run at once, in eight
// groups of 16 or more SMs with one block on each (two at d = 64 and up to 8 heads); the larger
// the sooner they are done. Where they do not fit, a warp does 16 tiles in about the time that
// the plan and the join take.
int decode_team(int items, double tiles, int d, int heads) {
  if (tiles <= 8) return 0;
  const int each = d == 64 && heads <= 8 ? 2 : 1;
  for (int team = kTeamBlocks; team >= 1; team /= 2)
    if (tiles <= 8 * kTeamWarps * team && (double)items * team <= 128 * each) return team;
  return tiles <= 16 ? 0 : -1;
}

// Items of a group, `lanes` threads to an item. The plan's cluster has room for kPlanBlocks *
// kPlanThreads groups: one item each while they last, which it describes itself; else whole rounds
// of a block of decode_walks_kernel, so that no block describes an item of another's group.
int decode_group(long long items, int lanes) {
  const long long most = (long long)kPlanBlocks * kPlanThreads, round = kWalkThreads / lanes;
  return items <= most ? 1 : (int)(round * ((items + round * most - 1) / (round * most)));
}

// The kernels that a call takes, and how they share its items.
struct DecodeRoute {
  int team;                // blocks of a team in decode_team_kernel; 0: a warp for each item; -1: ranges
  bool dense;              // one pattern with r = 1
  bool grouped;            // several tokens to an item
  int walks;               // of an item: patterns, or tokens
  int heads, tokens, nsub, items, group, lanes, warps;  // as in DecodeParams
  bool plan_alone;         // the plan is one block
  bool join_items;         // the join has a block for each item
};
// `longest`: positions that the table has; of_seq: tokens name their sequences.
DecodeRoute decode_route(int T, int B, int Hkv, int G, int d, bool of_seq, const int* w, const int* r,
                         int npat, long long longest, int num_sms) {
  DecodeRoute a;
  a.dense = npat == 1 && r[0] == 1;
  // the most tiles that an item of one token can have, as far as the table goes
  double tiles = 0;
  for (int i = 0; i < npat; ++i) {
    const long long n = (std::min<long long>(w[i], longest) + r[i] - 1) / r[i];
    tiles += (double)((n + kDecTile - 1) / kDecTile);
  }
  a.team = decode_team((int)decode_items(T, Hkv, G, false), tiles, d, decode_heads(G, false));
  // Tokens of one sequence, which attention over all that it holds (one segment) takes together,
  // where the call has one and a half for each row of the table; while the weights of eight contexts
  // fit an int. Tokens that share no row only widen a tile: 32 ragged contexts up to 32768 of 8 KV
  // heads took (together | one by one) 116 | 94 us with 33 tokens, 118 | 114 with 40, 118 | 136 with
  // 48, 119 | 170 with 64 for one head of d = 64, and 199 | 159, 200 | 194, 200 | 234, 198 | 303 for
  // four of d = 128.
  a.grouped = a.team < 0 && a.dense && w[0] >= longest && of_seq && 2ll * T >= 3ll * B && G <= 8 &&
              longest < (1ll << 28);
  a.tokens = decode_tokens(G, a.grouped);
  a.walks = a.grouped ? a.tokens : npat;
  a.heads = decode_heads(G, a.grouped);
  a.nsub = a.grouped ? 1 : (G + a.heads - 1) / a.heads;
  a.items = (int)decode_items(T, Hkv, G, a.grouped);
  a.lanes = 1;
  while (a.lanes < a.walks) a.lanes *= 2;
  a.group = decode_group(a.items, a.lanes);
  // no more warps than have work
  const int blocks = std::min(num_sms, kDecMaxSms) * decode_blocks_per_sm(d, a.heads, a.grouped);
  a.warps = kDecWarps * (int)std::min<double>(blocks, std::max(tiles * a.tokens, 1.0) * a.items * kSpreadWeight /
                                                              (kDecWarps * kRangeWeight) + 1);
  // one block saves the cluster's barriers as long as it describes all items at once
  a.plan_alone = a.group == 1 && a.items <= kPlanAlone / a.lanes;
  // a block for each item while they are fewer than blocks for every eight ranges
  a.join_items = a.items <= (a.warps + kJoinWarps - 1) / kJoinWarps;
  return a;
}

// Workspace of a decode: the items' walks, the warps' ranges, and the partials of cut items.
struct DecodeScratch {
  size_t head, walk, upto, sums, range, part;
  size_t total() const { return head + walk + upto + sums + range + part; }
};
DecodeScratch decode_scratch(int T, int H, int Hkv, int d, bool grouped) {
  const int G = H / Hkv;
  const size_t items = (size_t)decode_items(T, Hkv, G, grouped);
  const size_t warps = (size_t)kDecMaxSms * decode_blocks_per_sm(d, decode_heads(G, grouped), grouped) * kDecWarps;
  DecodeScratch s;
  s.head = align256(items * sizeof(DecodeHead));
  s.walk = align256(items * kMaxPat * sizeof(DecodeWalk));
  s.upto = align256(items * 8);
  s.sums = align256((size_t)kPlanBlocks * kPlanThreads * 8);
  s.range = align256((warps + 1) * sizeof(DecodeRange));
  s.part = align256(warps * 2 * decode_columns(G, grouped) * (d + 4) * 4);
  return s;
}

template <int D, int HEADS, int FMT>
cudaError_t launch_decode(const DecodeParams& p, const DecodeRoute& a, cudaStream_t stream) {
  if (p.team >= 0) {
    const auto kernel = decode_team_kernel<D, HEADS, FMT>;
    const size_t smem = p.team == 0 ? 0 : (size_t)(kTeamWarps + 1) * p.part_stride * 4;
    // with the static part more than 48 KB; opting in (always to the same most, for calls of other
    // threads) is needed once per device and costs nothing to repeat
    if constexpr (HEADS * D >= 1024) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (kTeamWarps + 1) * HEADS * (D + 4) * 4);
      if (e != cudaSuccess) return e;
    }
    const dim3 grid((unsigned)(p.team == 0 ? (p.items + kTeamWarps - 1) / kTeamWarps : p.items * p.team));
    return launch_overlapped(kernel, grid, kTeamWarps * 32, smem, stream, std::max(p.team, 1), p);
  }
  const int groups = (int)(((long long)p.items + p.group - 1) / p.group);
  cudaError_t e = cudaSuccess;
  if (p.group > 1)
    e = launch_overlapped(decode_walks_kernel, dim3((unsigned)groups), kWalkThreads, 0, stream, 1, p);
  if (e == cudaSuccess)
    e = a.plan_alone
            ? launch_overlapped(decode_plan_kernel<1>, dim3(1), kPlanAlone, 0, stream, 1, p)
            : launch_overlapped(decode_plan_kernel<kPlanBlocks>, dim3(kPlanBlocks), kPlanThreads, 0, stream,
                                kPlanBlocks, p);
  if (e != cudaSuccess) return e;
  auto kernel = p.dense ? decode_kernel<D, HEADS, FMT, kDense> : decode_kernel<D, HEADS, FMT, kAnyPatterns>;
  if constexpr (HEADS >= 8)
    if (p.tokens > 1) kernel = decode_kernel<D, HEADS, FMT, kGrouped>;
  e = launch_overlapped(kernel, dim3((unsigned)(p.warps / kDecWarps)), kDecWarps * 32, 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  const int by_ranges = (p.warps + kJoinWarps - 1) / kJoinWarps;
  return launch_overlapped(a.join_items ? decode_join_items_kernel<D> : decode_join_ranges_kernel<D>,
                           dim3((unsigned)(a.join_items ? p.items : by_ranges), (unsigned)p.part_heads), kJoinThreads,
                           0, stream, 1, p);
}
template <int D, int FMT>
cudaError_t launch_decode_heads(const DecodeParams& p, const DecodeRoute& a, cudaStream_t stream) {
  switch (p.heads) {
    case 1: return launch_decode<D, 1, FMT>(p, a, stream);
    case 2: return launch_decode<D, 2, FMT>(p, a, stream);
    case 4: return launch_decode<D, 4, FMT>(p, a, stream);
    case 8: return launch_decode<D, 8, FMT>(p, a, stream);
    default: return launch_decode<D, 16, FMT>(p, a, stream);
  }
}

// Inverse of an odd number modulo 2^32: Newton's step doubles the correct low bits.
uint32_t odd_inverse(uint32_t x) {
  uint32_t y = x;  // right to 3 bits
  for (int i = 0; i < 4; ++i) y *= 2u - x * y;
  return y;
}

// The patterns by ascending r, with the constants of their divisions.
void decode_patterns(DecodeParams& p, const int* w, const int* r, int npat) {
  int order[kMaxPat];
  for (int i = 0; i < npat; ++i) order[i] = i;
  std::stable_sort(order, order + npat, [&](int a, int b) { return r[a] < r[b]; });
  for (int i = 0; i < npat; ++i) {
    p.w[i] = w[order[i]];
    p.r[i] = r[order[i]];
    divisor_magic((uint32_t)p.w[i], p.w_mul[i], p.w_sh[i]);
    divisor_magic((uint32_t)p.r[i], p.r_mul[i], p.r_sh[i]);
    uint32_t odd = (uint32_t)p.r[i];
    while ((odd & 1u) == 0) {
      odd >>= 1;
      ++p.r_rot[i];
    }
    p.r_inv[i] = odd_inverse(odd);
    p.r_lim[i] = 0xffffffffu / (uint32_t)p.r[i];
    for (int l = 0; l < i; ++l)
      if (p.r[i] % p.r[l] == 0) p.divisors[i] |= 1u << l;
  }
}

}  // namespace
}  // namespace dil

extern "C" size_t dilattn_decode_workspace_size(int T, int H, int Hkv, int d) {
  if (T < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || (d != 64 && d != 128)) return 0;
  const size_t plain = decode_scratch(T, H, Hkv, d, false).total();
  return T > 1 && H / Hkv <= 8 ? std::max(plain, decode_scratch(T, H, Hkv, d, true).total()) : plain;
}

extern "C" int dilattn_decode(const void* q, long long q_stride, const void* kc, const void* vc,
                              const float* ks, const float* vs, int pages, int Hkv, int page_size,
                              int d, int format, const int* table, int B, int max_pages,
                              const int* seq, const int* pos, void* out, float* lse, int T, int H,
                              const int* w, const int* r, int npat, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_cache(kc, vc, ks, vs, pages, Hkv, page_size, d, format, table, B, max_pages);
  if (rc != DILATTN_OK) return rc;
  if (T < 0 || H < 1 || H % Hkv != 0 || (seq == nullptr && T > B)) return DILATTN_ERR_INVALID_ARG;
  if (npat < 1 || npat > DILATTN_MAX_PATTERNS || w == nullptr || r == nullptr)
    return DILATTN_ERR_INVALID_ARG;
  for (int i = 0; i < npat; ++i)
    if (w[i] < 1 || r[i] < 1) return DILATTN_ERR_INVALID_ARG;
  if (!good_stride(q_stride, (long long)H * d) || (seq != nullptr && !aligned4(seq)))
    return DILATTN_ERR_INVALID_ARG;
  if ((double)T * H * d >= 1099511627776.0 || (double)T * H > 2147483647.0)
    return DILATTN_ERR_INVALID_ARG;
  if (T == 0) return DILATTN_OK;
  if (!aligned16(q) || !aligned16(out) || !aligned4(pos) || (lse != nullptr && !aligned16(lse)))
    return DILATTN_ERR_INVALID_ARG;
  const size_t need = dilattn_decode_workspace_size(T, H, Hkv, d);
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 ||
      workspace_bytes < need)
    return DILATTN_ERR_WORKSPACE;
  const size_t cb = (size_t)pages * Hkv * page_size * d, sb = (size_t)pages * Hkv * 4;
  const Span mut[3] = {{out, (size_t)T * H * d * 2},
                       {workspace, need},
                       {lse, lse != nullptr ? (size_t)T * H * 4 : 0}};
  const Span ro[8] = {{kc, cb}, {vc, cb}, {ks, sb}, {vs, sb},
                      {table, (size_t)B * max_pages * 4},
                      {q, strided_bytes(T, (long long)H * d, q_stride)},
                      {pos, (size_t)T * 4},
                      {seq, seq != nullptr ? (size_t)T * 4 : 0}};
  if (any_overlap(mut, 3, ro, 8) || any_overlap(mut, 1, mut + 1, 2) ||
      any_overlap(mut + 1, 1, mut + 2, 1))
    return DILATTN_ERR_INVALID_ARG;
  DeviceState* st = nullptr;
  rc = device_state(&st);
  if (rc != DILATTN_OK) return rc;
  NvtxRange range("dilattn decode");
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  p.geom = cache_geom(table, B, max_pages, pages, Hkv, page_size, st);
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.codes[0] = reinterpret_cast<const uint8_t*>(kc);
  p.codes[1] = reinterpret_cast<const uint8_t*>(vc);
  p.scale[0] = ks;
  p.scale[1] = vs;
  p.seq = seq;
  p.pos = pos;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.T = T;
  p.H = H;
  p.qk_scale = (float)(1.4426950408889634 / std::sqrt((double)d));
  decode_patterns(p, w, r, npat);
  p.G = H / Hkv;
  const DecodeRoute a = decode_route(T, B, Hkv, p.G, d, seq != nullptr, w, r, npat,
                                     (long long)max_pages * page_size, st->num_sms);
  p.team = a.team;
  p.dense = a.dense;
  p.tokens = a.tokens;
  p.g_rec = (256 + p.G - 1) / p.G;
  if (a.grouped)
    for (int i = 0; i < a.walks; ++i) p.r[i] = 1;
  p.npat = a.walks;
  p.heads = a.heads;
  p.nsub = a.nsub;
  p.per_token = Hkv * p.nsub;
  divisor_magic((uint32_t)p.per_token, p.pt_mul, p.pt_sh);
  divisor_magic((uint32_t)p.nsub, p.ns_mul, p.ns_sh);
  p.items = a.items;
  p.lanes = a.lanes;
  p.group = a.group;
  p.warps = a.warps;
  const DecodeScratch lay = decode_scratch(T, H, Hkv, d, a.grouped);
  char* at = reinterpret_cast<char*>(workspace);
  auto take = [&at](size_t n) { return at += n, at - n; };
  p.head = reinterpret_cast<DecodeHead*>(take(lay.head));
  p.walk = reinterpret_cast<DecodeWalk*>(take(lay.walk));
  p.upto = reinterpret_cast<long long*>(take(lay.upto));
  p.sums = reinterpret_cast<long long*>(take(lay.sums));
  p.range = reinterpret_cast<DecodeRange*>(take(lay.range));
  p.part = reinterpret_cast<float*>(take(lay.part));
  p.part_heads = decode_columns(p.G, a.grouped);
  p.part_stride = p.part_heads * (d + 4);
  cudaError_t e;
  if (format == DILATTN_CACHE_E4M3)
    e = d == 64 ? launch_decode_heads<64, kFmtE4M3>(p, a, stream) : launch_decode_heads<128, kFmtE4M3>(p, a, stream);
  else
    e = d == 64 ? launch_decode_heads<64, kFmtInt8>(p, a, stream) : launch_decode_heads<128, kFmtInt8>(p, a, stream);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  return DILATTN_OK;
}
