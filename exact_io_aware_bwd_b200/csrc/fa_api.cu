// Host side of libfa_b200.so: argument checks, TMA tensor maps and kernel
// launches behind the C ABI declared in include/fa.h.  The whole library is
// this one translation unit (the kernels are included below).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <utility>

#include "fa.h"
#include "sm100.cuh"
#include "fa_fwd.cuh"
#include "fa_fwd_fp8.cuh"
#include "fa_bwd.cuh"
#include "fa_decode.cuh"
#include "fa_append.cuh"
#include "fa_paged.cuh"
#include "fa_prefix.cuh"

// The kernel ids in the status word say which kernel recorded an error.
namespace fa {
constexpr uint32_t kKernelIds[] = {kKernFwd, kKernBwdPre, kKernBwd, kKernBwdPost, kKernSelftest, kKernDecode,
                                   kKernDecodeMerge, kKernFwdFp8, kKernPaged, kKernPrefixOwn, kKernAppend};
constexpr bool ids_differ() {
  for (const uint32_t& a : kKernelIds)
    for (const uint32_t& b : kKernelIds)
      if (&a != &b && a == b) return false;
  return true;
}
static_assert(ids_differ(), "two kernels share an id");
}  // namespace fa

namespace {

using fa::FwdLayout;
using fa::FwdParams;

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// 3-D tiled map over a dense [outer][rows][cols] tensor (cols contiguous),
// copied in boxes of box_rows x box_cols with 128-byte swizzle.  Out-of-range
// rows read as zero and are skipped on stores.
bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, uint64_t cols,
              uint64_t rows, uint64_t outer, uint32_t box_cols, uint32_t box_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {cols, rows, outer};
  cuuint64_t strides[2] = {cols * esize, cols * rows * esize};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Events bracketing the launches of one kernel (see fa_set_profile_events).
cudaEvent_t g_prof_start[8] = {nullptr};
cudaEvent_t g_prof_stop[8] = {nullptr};

void prof_begin(int id, cudaStream_t st) {
  if (g_prof_start[id]) cudaEventRecord(g_prof_start[id], st);
}
void prof_end(int id, cudaStream_t st) {
  if (g_prof_stop[id]) cudaEventRecord(g_prof_stop[id], st);
}

// Cap on the persistent blocks of the backward main pass (0: one per SM).
std::atomic<int> g_bwd_max_blocks{0};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device must be sm_100 (B200 class); checked once per device.
fa_status_t check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  static std::atomic<int> ok_dev[64] = {};  // 0 unknown, 1 ok, 2 not ok (calls may race)
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  if (ok_dev[dev].load() == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return FA_ERR_CUDA;
    ok_dev[dev].store((major == 10 && minor == 0) ? 1 : 2);
  }
  return ok_dev[dev].load() == 1 ? FA_OK : FA_ERR_UNSUPPORTED;
}

// Number of SMs of the current device (cached per device); 0 on error.
int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  static std::atomic<int> n_sm[64] = {};  // 0: not yet queried (calls may race)
  if (n_sm[dev].load() == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    n_sm[dev].store(n);
  }
  return n_sm[dev].load();
}

// Dropout probability -> 8-bit threshold t = round(256 p): a key is dropped
// when its random byte is below t.  p must be finite, 0 <= p and t <= 255.
bool drop_threshold(float p, int* t) {
  if (!std::isfinite(p) || p < 0.f) return false;
  const long r = std::lround(static_cast<double>(p) * 256.0);
  if (r > 255) return false;
  *t = static_cast<int>(r);
  return true;
}

// Checks shared by fa_fwd and fa_bwd.  Sets *empty for a problem with no work.
fa_status_t check_common(int B, int Hq, int Hkv, int N, int d, float scale, int causal,
                         fa_dtype_t dtype, bool* empty) {
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0) return FA_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // sizes the kernels index with 32-bit block counts and TMA coordinates
  const int64_t tiles = (static_cast<int64_t>(N) + 127) / 128;
  if (static_cast<int64_t>(B) * Hq * tiles > INT32_MAX) return FA_ERR_UNSUPPORTED;
  *empty = (B == 0 || N == 0);
  return FA_OK;
}

// Opt a kernel into `smem` bytes of dynamic shared memory, once per kernel
// and device (the attribute belongs to the device's context).
template <typename K>
fa_status_t opt_in_smem(K kernel, int smem) {
  static std::mutex mu;
  static const void* done_fn[256];
  static int done_dev[256];
  static int n_done = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_done; ++i)
    if (done_fn[i] == reinterpret_cast<const void*>(kernel) && done_dev[i] == dev) return FA_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return FA_ERR_CUDA;
  if (n_done < 256) {
    done_fn[n_done] = reinterpret_cast<const void*>(kernel);
    done_dev[n_done++] = dev;
  }
  return FA_OK;
}

// Launches `kernel` as a programmatic dependent of the kernel before it on the
// stream: it may be scheduled while that kernel still runs, and waits
// (griddepcontrol.wait) before it touches global memory.  Used on the serving
// path (cache append, decode), whose launch gaps are a visible part of a step;
// on the training path it measured slower and is not used.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned block, int smem,
                             cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int HD, bool BF, bool CA, bool DR, bool BM = false>
fa_status_t launch_fwd(const FwdParams& prm, cudaStream_t st) {
  auto kern = fa::fa_fwd_kernel<HD, BF, CA, DR, BM>;
  const int smem = FwdLayout<HD>::kDynSmem;
  fa_status_t s = opt_in_smem(kern, smem);
  if (s != FA_OK) return s;
  // one block per (head, couple of query pairs) or per (head, query pair)
  const int grid = (prm.fold ? (prm.n_pairs + 1) / 2 : prm.n_pairs) * prm.BH;
  prof_begin(fa::kKernFwd, st);
  kern<<<grid, fa::kFwdThreads, smem, st>>>(prm);
  const bool ok = cudaGetLastError() == cudaSuccess;
  prof_end(fa::kKernFwd, st);
  return ok ? FA_OK : FA_ERR_CUDA;
}

template <int HD, bool BF>
fa_status_t launch_fwd_c(const FwdParams& prm, int causal, cudaStream_t st) {
  if (prm.bmask != nullptr)
    return causal ? launch_fwd<HD, BF, true, false, true>(prm, st) : launch_fwd<HD, BF, false, false, true>(prm, st);
  if (prm.drop_t > 0)
    return causal ? launch_fwd<HD, BF, true, true>(prm, st) : launch_fwd<HD, BF, false, true>(prm, st);
  return causal ? launch_fwd<HD, BF, true, false>(prm, st) : launch_fwd<HD, BF, false, false>(prm, st);
}

// The FP8 forward kernel; its launches are bracketed by the forward's
// profiling events.
template <bool OB, bool CA>
fa_status_t launch_fwd_fp8(const fa::Fp8FwdParams& prm, cudaStream_t st) {
  auto kern = fa::fa_fwd_fp8_kernel<OB, CA>;
  const int smem = fa::Fp8FwdLayout::kDynSmem;
  fa_status_t s = opt_in_smem(kern, smem);
  if (s != FA_OK) return s;
  // one block per (head, couple of query pairs) or per (head, query pair)
  const int grid = (prm.fold ? (prm.n_pairs + 1) / 2 : prm.n_pairs) * prm.BH;
  prof_begin(fa::kKernFwd, st);
  kern<<<grid, fa::kFwdFp8Threads, smem, st>>>(prm);
  const bool ok = cudaGetLastError() == cudaSuccess;
  prof_end(fa::kKernFwd, st);
  return ok ? FA_OK : FA_ERR_CUDA;
}

template <int HD, bool BF, bool CA, bool DR, bool BM = false>
fa_status_t launch_bwd_main(const fa::BwdParams& prm, int grid, cudaStream_t st) {
  auto kern = fa::fa_bwd_kernel<HD, BF, CA, DR, BM>;
  const int smem = fa::BwdLayout<HD>::kDynSmem;
  fa_status_t s = opt_in_smem(kern, smem);
  if (s != FA_OK) return s;
  prof_begin(fa::kKernBwd, st);
  kern<<<grid, fa::kBwdThreads, smem, st>>>(prm);
  const bool ok = cudaGetLastError() == cudaSuccess;
  prof_end(fa::kKernBwd, st);
  return ok ? FA_OK : FA_ERR_CUDA;
}

template <int HD, bool BF>
fa_status_t bwd_run(const void* q, const void* k, const void* v, const void* o, const void* dout,
                    const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                    float scale, int causal, int window, uint32_t drop_t, uint64_t seed,
                    void* workspace, cudaStream_t st, const uint8_t* bmask = nullptr,
                    long long bm_hstride = 0) {
  const int64_t Np = fa::bwd_padded_rows(N);
  const int64_t BHq = static_cast<int64_t>(B) * Hq, BHkv = static_cast<int64_t>(B) * Hkv;
  float* Dvec = static_cast<float*>(workspace);
  float* lse2 = Dvec + BHq * Np;
  float* dqacc = lse2 + BHq * Np;
  const int64_t rows = BHq * Np;
  unsigned* work_counter = reinterpret_cast<unsigned*>(dqacc + rows * HD);
  const int n_ktiles = (N + 127) / 128;

  // 1. D, lse2, zeroed accumulator and work counter
  fa::BwdPreParams pre;
  std::memset(&pre, 0, sizeof(pre));
  pre.o = o;
  pre.dout = dout;
  pre.lse = lse;
  pre.Dvec = Dvec;
  pre.lse2 = lse2;
  pre.dqacc = dqacc;
  pre.work_counter = work_counter;
  pre.N = N;
  pre.Np = static_cast<int>(Np);
  pre.total_rows = rows;
  {
    // HD / 8 threads a row; a grid of 16 blocks of 256 threads per SM, each
    // thread taking rows in turn
    const int64_t groups = rows * (HD / 8);
    int n_sm = sm_count();
    if (n_sm <= 0) return FA_ERR_CUDA;
    const int64_t blocks = std::min<int64_t>((groups + 255) / 256, static_cast<int64_t>(n_sm) * 16);
    fa::fa_bwd_pre_kernel<HD, BF><<<static_cast<unsigned>(blocks), 256, 0, st>>>(pre);
  }
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;

  // 1b. block mask: the walk of every work item
  uint16_t* plan_list = nullptr;
  int* plan_steps = nullptr;
  const int plan_cap = (Hq / Hkv) * n_ktiles;
  if (bmask != nullptr) {
    plan_steps = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(workspace) + fa::bwd_workspace_bytes(B, Hq, N, HD));
    plan_list = reinterpret_cast<uint16_t*>(plan_steps + BHkv * n_ktiles);
    fa::BwdPlanParams pl;
    std::memset(&pl, 0, sizeof(pl));
    pl.bmask = bmask;
    pl.bm_hstride = bm_hstride;
    pl.list = plan_list;
    pl.steps = plan_steps;
    pl.N = N;
    pl.Hq = Hq;
    pl.Hkv = Hkv;
    pl.group = Hq / Hkv;
    pl.n_ktiles = n_ktiles;
    pl.n_qtiles = (N + 63) / 64;
    pl.causal = causal;
    pl.window = window;
    pl.cap = plan_cap;
    pl.n_items = static_cast<int>(BHkv * n_ktiles);
    fa::fa_bwd_plan_kernel<<<static_cast<unsigned>((pl.n_items + 7) / 8), 256, 0, st>>>(pl);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  }

  // 2. main pass
  const CUtensorMapDataType dt = BF ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  fa::BwdParams prm;
  std::memset(&prm, 0, sizeof(prm));
  if (!make_map(&prm.tm_q, q, dt, 2, HD, N, BHq, 64, 64) ||
      !make_map(&prm.tm_do, dout, dt, 2, HD, N, BHq, 64, 64) ||
      !make_map(&prm.tm_k, k, dt, 2, HD, N, BHkv, 64, 128) ||
      !make_map(&prm.tm_v, v, dt, 2, HD, N, BHkv, 64, 128))
    return FA_ERR_CUDA;
  prm.lse2 = lse2;
  prm.Dvec = Dvec;
  prm.dqacc = dqacc;
  prm.plan_list = plan_list;
  prm.plan_steps = plan_steps;
  prm.plan_cap = plan_cap;
  prm.dk = dk;
  prm.dv = dv;
  prm.work_counter = work_counter;
  prm.N = N;
  prm.Np = static_cast<int>(Np);
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.group = Hq / Hkv;
  prm.n_ktiles = (N + 127) / 128;
  prm.n_qtiles = (N + 63) / 64;
  prm.BHkv = static_cast<int>(BHkv);
  prm.scale = scale;
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  prm.window = window;
  prm.drop_t = drop_t;
  prm.drop_scale = drop_t ? 256.0f / static_cast<float>(256u - drop_t) : 1.0f;
  prm.seed_lo = static_cast<uint32_t>(seed);
  prm.seed_hi = static_cast<uint32_t>(seed >> 32);
  prm.n_items = prm.n_ktiles * prm.BHkv;
  {
    // kv heads per chunk of the item order: Q, dO (group query heads), K, V
    // and the fp32 dQ accumulator of a chunk stay within about 48 MB of L2
    const double head_bytes = static_cast<double>(prm.group) * N * HD * 2.0 * 2.0 +
                              static_cast<double>(prm.group) * Np * HD * 4.0 +
                              static_cast<double>(N) * HD * 2.0 * 2.0;
    const double c = std::floor(48.0 * 1024.0 * 1024.0 / head_bytes);
    prm.chunk_heads = static_cast<int>(std::max(1.0, std::min(c, static_cast<double>(prm.BHkv))));
  }
  int n_sm = 0;
  if ((n_sm = sm_count()) <= 0) return FA_ERR_CUDA;
  const int cap = g_bwd_max_blocks.load();
  const int grid = std::min(prm.n_items, cap > 0 ? std::min(cap, n_sm) : n_sm);  // persistent
  fa_status_t s;
  if (bmask != nullptr)
    s = causal ? launch_bwd_main<HD, BF, true, false, true>(prm, grid, st)
               : launch_bwd_main<HD, BF, false, false, true>(prm, grid, st);
  else if (prm.drop_t > 0)
    s = causal ? launch_bwd_main<HD, BF, true, true>(prm, grid, st)
               : launch_bwd_main<HD, BF, false, true>(prm, grid, st);
  else
    s = causal ? launch_bwd_main<HD, BF, true, false>(prm, grid, st)
               : launch_bwd_main<HD, BF, false, false>(prm, grid, st);
  if (s != FA_OK) return s;

  // 3. dQ = scale * accumulator
  const int64_t total_vec = BHq * N * (HD / 8);
  const int64_t blocks = std::min<int64_t>((total_vec + 255) / 256, 148 * 16);
  fa::fa_bwd_post_kernel<HD, BF><<<static_cast<unsigned>(blocks), 256, 0, st>>>(
      dqacc, dq, N, static_cast<int>(Np), total_vec, scale);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

}  // extern "C"

namespace {

fa_status_t fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int Hq, int Hkv, int N, int d, float scale, int causal, int window,
                     uint32_t drop_t, uint64_t seed, fa_dtype_t dtype, void* stream,
                     const uint8_t* bmask = nullptr, long long bm_hstride = 0) {
  bool empty = false;
  fa_status_t s = check_common(B, Hq, Hkv, N, d, scale, causal, dtype, &empty);
  if (s != FA_OK) return s;
  if (empty) return FA_OK;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_MISALIGNED;
  if ((s = check_device()) != FA_OK) return s;

  const bool bf = dtype == FA_BF16;
  const CUtensorMapDataType dt = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  FwdParams prm;
  std::memset(&prm, 0, sizeof(prm));
  const uint64_t BHq = static_cast<uint64_t>(B) * Hq, BHkv = static_cast<uint64_t>(B) * Hkv;
  if (!make_map(&prm.tm_q, q, dt, 2, d, N, BHq, 64, 128) ||
      !make_map(&prm.tm_k, k, dt, 2, d, N, BHkv, 64, 128) ||
      !make_map(&prm.tm_v, v, dt, 2, d, N, BHkv, 64, 128))
    return FA_ERR_CUDA;
  prm.o = o;
  prm.lse = lse;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.group = Hq / Hkv;
  prm.BH = static_cast<int>(BHq);
  prm.n_pairs = (N + 255) / 256;
  // fold two query pairs into a block while a pair is short (its fixed costs
  // then weigh most): up to 64 pairs (N <= 16384)
  prm.fold = prm.n_pairs <= 64 ? 1 : 0;
  prm.n_ktiles = (N + 127) / 128;
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  prm.window = window;
  prm.drop_t = drop_t;
  prm.drop_scale = drop_t ? 256.0f / static_cast<float>(256u - drop_t) : 1.0f;
  prm.seed_lo = static_cast<uint32_t>(seed);
  prm.seed_hi = static_cast<uint32_t>(seed >> 32);
  prm.bmask = bmask;
  prm.bm_hstride = bm_hstride;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d == 128) return bf ? launch_fwd_c<128, true>(prm, causal, st) : launch_fwd_c<128, false>(prm, causal, st);
  return bf ? launch_fwd_c<64, true>(prm, causal, st) : launch_fwd_c<64, false>(prm, causal, st);
}

}  // namespace

extern "C" {

fa_status_t fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                   int Hq, int Hkv, int N, int d, float scale, int causal, fa_dtype_t dtype,
                   void* stream) {
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, 0, 0, 0, dtype, stream);
}

fa_status_t fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                          int Hq, int Hkv, int N, int d, float scale, int window, fa_dtype_t dtype,
                          void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, 1, window, 0, 0, dtype, stream);
}

fa_status_t fa_fwd_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                           int Hq, int Hkv, int N, int d, float scale, int causal, float p_drop,
                           uint64_t seed, fa_dtype_t dtype, void* stream) {
  int t = 0;
  if (!drop_threshold(p_drop, &t)) return FA_ERR_INVALID_ARG;
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, 0, static_cast<uint32_t>(t),
                  seed, dtype, stream);
}

fa_status_t fa_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int Hq, int Hkv, int N, int d, float scale, float descale_q,
                       float descale_k, float descale_v, int causal, fa_dtype_t out_dtype,
                       void* stream) {
  bool empty = false;
  fa_status_t s = check_common(B, Hq, Hkv, N, d, scale, causal, out_dtype, &empty);
  if (s != FA_OK) return s;
  for (float f : {descale_q, descale_k, descale_v})
    if (!std::isfinite(f) || !(f > 0.f)) return FA_ERR_INVALID_ARG;
  const double c = static_cast<double>(scale) * descale_q * descale_k * 1.4426950408889634;
  if (!(c >= 1.2e-38) || c > 3.0e38) return FA_ERR_INVALID_ARG;  // a normal fp32 factor
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (empty) return FA_OK;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_MISALIGNED;
  if ((s = check_device()) != FA_OK) return s;

  const bool bf = out_dtype == FA_BF16;
  const CUtensorMapDataType dt16 = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  fa::Fp8FwdParams prm;
  std::memset(&prm, 0, sizeof(prm));
  const uint64_t BHq = static_cast<uint64_t>(B) * Hq, BHkv = static_cast<uint64_t>(B) * Hkv;
  if (!make_map(&prm.tm_q, q, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, N, BHq, 128, 128) ||
      !make_map(&prm.tm_k, k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, N, BHkv, 128, 128) ||
      !make_map(&prm.tm_v, v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, N, BHkv, 128, 128) ||
      !make_map(&prm.tm_o, o, dt16, 2, 128, N, BHq, 64, 128))
    return FA_ERR_CUDA;
  prm.lse = lse;
  prm.N = N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.group = Hq / Hkv;
  prm.BH = static_cast<int>(BHq);
  prm.n_pairs = (N + 255) / 256;
  prm.fold = prm.n_pairs <= 64 ? 1 : 0;  // as in the 16-bit forward
  prm.n_ktiles = (N + 127) / 128;
  prm.scale_log2 = static_cast<float>(c);
  prm.delta_v = descale_v;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (causal) return bf ? launch_fwd_fp8<true, true>(prm, st) : launch_fwd_fp8<false, true>(prm, st);
  return bf ? launch_fwd_fp8<true, false>(prm, st) : launch_fwd_fp8<false, false>(prm, st);
}

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0) return 0;
  return fa::bwd_workspace_bytes(B, Hq, N, d);
}

}  // extern "C"

namespace {

// Block-mask additions to the backward workspace: the step count and the
// walk of every work item (see fa_bwd_plan_kernel).
size_t bwd_mask_plan_bytes(int B, int Hq, int Hkv, int N) {
  const int64_t n_ktiles = (static_cast<int64_t>(N) + 127) / 128;
  const int64_t items = static_cast<int64_t>(B) * Hkv * n_ktiles;
  const int64_t cap = static_cast<int64_t>(Hq / Hkv) * n_ktiles;
  return static_cast<size_t>(items) * 4u + static_cast<size_t>(items * cap) * 2u;
}

// Sizes a block mask supports: the walk entries hold the group head in 4
// bits and the query block in 12.
bool bmask_supported(int Hq, int Hkv, int N) {
  return Hq / Hkv <= 16 && (static_cast<int64_t>(N) + 127) / 128 <= 4096;
}

fa_status_t bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                     int d, float scale, int causal, int window, uint32_t drop_t, uint64_t seed,
                     fa_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream,
                     const uint8_t* bmask = nullptr, long long bm_hstride = 0) {
  bool empty = false;
  fa_status_t s = check_common(B, Hq, Hkv, N, d, scale, causal, dtype, &empty);
  if (s != FA_OK) return s;
  if (empty) return FA_OK;
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace)
    return FA_ERR_INVALID_ARG;
  size_t need = fa::bwd_workspace_bytes(B, Hq, N, d);
  if (bmask != nullptr) {
    if (!bmask_supported(Hq, Hkv, N)) return FA_ERR_UNSUPPORTED;
    need += bwd_mask_plan_bytes(B, Hq, Hkv, N);
  }
  if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
      !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(workspace))
    return FA_ERR_MISALIGNED;
  if ((s = check_device()) != FA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == FA_BF16;
  if (d == 128)
    return bf ? bwd_run<128, true>(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, scale, causal, window, drop_t, seed, workspace, st, bmask, bm_hstride)
              : bwd_run<128, false>(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, scale, causal, window, drop_t, seed, workspace, st, bmask, bm_hstride);
  return bf ? bwd_run<64, true>(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, scale, causal, window, drop_t, seed, workspace, st, bmask, bm_hstride)
            : bwd_run<64, false>(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, scale, causal, window, drop_t, seed, workspace, st, bmask, bm_hstride);
}

}  // namespace

extern "C" {

fa_status_t fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                   const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                   int d, float scale, int causal, fa_dtype_t dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, 0, 0, 0,
                  dtype, workspace, workspace_bytes, stream);
}

fa_status_t fa_bwd_window(const void* q, const void* k, const void* v, const void* o,
                          const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                          int Hq, int Hkv, int N, int d, float scale, int window, fa_dtype_t dtype,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 1) return FA_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, 1, window, 0, 0,
                  dtype, workspace, workspace_bytes, stream);
}

fa_status_t fa_bwd_dropout(const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                           int Hq, int Hkv, int N, int d, float scale, int causal, float p_drop,
                           uint64_t seed, fa_dtype_t dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int t = 0;
  if (!drop_threshold(p_drop, &t)) return FA_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, 0,
                  static_cast<uint32_t>(t), seed, dtype, workspace, workspace_bytes, stream);
}

fa_status_t fa_fwd_blockmask(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                             int Hq, int Hkv, int N, int d, float scale, int causal,
                             const uint8_t* block_mask, int mask_per_head, fa_dtype_t dtype,
                             void* stream) {
  if (block_mask == nullptr || (mask_per_head != 0 && mask_per_head != 1)) return FA_ERR_INVALID_ARG;
  if (Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && !bmask_supported(Hq, Hkv, N)) return FA_ERR_UNSUPPORTED;
  const long long nb = (static_cast<long long>(N) + 127) / 128;
  return fwd_impl(q, k, v, o, lse, B, Hq, Hkv, N, d, scale, causal, 0, 0, 0, dtype, stream, block_mask,
                  mask_per_head ? nb * nb : 0);
}

size_t fa_bwd_blockmask_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || Hq % Hkv != 0) return 0;
  return fa::bwd_workspace_bytes(B, Hq, N, d) + bwd_mask_plan_bytes(B, Hq, Hkv, N);
}

fa_status_t fa_bwd_blockmask(const void* q, const void* k, const void* v, const void* o,
                             const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                             int Hq, int Hkv, int N, int d, float scale, int causal,
                             const uint8_t* block_mask, int mask_per_head, fa_dtype_t dtype,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (block_mask == nullptr || (mask_per_head != 0 && mask_per_head != 1)) return FA_ERR_INVALID_ARG;
  const long long nb = (static_cast<long long>(N) + 127) / 128;
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, 0, 0, 0, dtype,
                  workspace, workspace_bytes, stream, block_mask, mask_per_head ? nb * nb : 0);
}

fa_status_t fa_get_device_status(void* stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return FA_ERR_CUDA;
  uint32_t word = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&word, fa::g_device_status, sizeof(word)) != cudaSuccess)
    return FA_ERR_CUDA;
  if (word == 0) return FA_OK;
  if (cudaMemcpyToSymbol(fa::g_device_status, &zero, sizeof(zero)) != cudaSuccess)
    return FA_ERR_CUDA;
  const uint32_t code = word & 0xFFu;
  if (code == fa::kStatusTimeout) return FA_ERR_TIMEOUT;
  if (code == fa::kStatusBadInput) return FA_ERR_INVALID_ARG;
  return FA_ERR_CUDA;
}

uint32_t fa_peek_device_status_word(void* stream) {
  cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  uint32_t word = 0;
  cudaMemcpyFromSymbol(&word, fa::g_device_status, sizeof(word));
  return word;
}

fa_status_t fa_selftest_wait_timeout(uint64_t limit_ns, void* stream) {
  fa_status_t s = check_device();
  if (s != FA_OK) return s;
  if (limit_ns == 0 || limit_ns > 10ull * 1000 * 1000 * 1000) return FA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // clear any earlier status, shorten the limit, run, restore
  if ((s = fa_get_device_status(stream)) == FA_ERR_CUDA) return s;
  const uint64_t dflt = 2000000000ull;
  if (cudaMemcpyToSymbolAsync(fa::g_wait_limit_ns, &limit_ns, sizeof(limit_ns), 0,
                              cudaMemcpyHostToDevice, st) != cudaSuccess)
    return FA_ERR_CUDA;
  fa::wait_timeout_selftest_kernel<<<1, 32, 0, st>>>();
  const bool launched = cudaGetLastError() == cudaSuccess;
  cudaMemcpyToSymbolAsync(fa::g_wait_limit_ns, &dflt, sizeof(dflt), 0, cudaMemcpyHostToDevice, st);
  if (!launched) return FA_ERR_CUDA;
  return fa_get_device_status(stream);
}

fa_status_t fa_set_profile_events(int kernel_id, void* start, void* stop) {
  if (kernel_id != static_cast<int>(fa::kKernFwd) && kernel_id != static_cast<int>(fa::kKernBwd))
    return FA_ERR_INVALID_ARG;
  if ((start == nullptr) != (stop == nullptr)) return FA_ERR_INVALID_ARG;
  g_prof_start[kernel_id] = reinterpret_cast<cudaEvent_t>(start);
  g_prof_stop[kernel_id] = reinterpret_cast<cudaEvent_t>(stop);
  return FA_OK;
}

size_t fa_decode_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int max_pages) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || d <= 0 || max_pages <= 0) return 0;
  return fa::decode_workspace_bytes(B, Hq, Hkv, Nq, d, max_pages);
}

fa_status_t fa_decode_paged(const void* q, const void* k_cache, const void* v_cache,
                            const int* block_table, const int* seq_lens, void* o, float* lse, int B,
                            int Hq, int Hkv, int Nq, int d, int page_size, int max_pages,
                            int num_pages, float scale, fa_dtype_t dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Nq <= 0 || max_pages <= 0 ||
      num_pages <= 0)
    return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return FA_ERR_UNSUPPORTED;
  if ((Hq / Hkv) * Nq > fa::kDecodeMaxRows) return FA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o || !lse || !workspace)
    return FA_ERR_INVALID_ARG;
  if (workspace_bytes < fa::decode_workspace_bytes(B, Hq, Hkv, Nq, d, max_pages))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u))
    return FA_ERR_MISALIGNED;
  fa_status_t s = check_device();
  if (s != FA_OK) return s;
  fa::DecodeParams prm;
  std::memset(&prm, 0, sizeof(prm));
  prm.q = q;
  prm.table = block_table;
  prm.lens = seq_lens;
  prm.o = o;
  prm.lse = lse;
  prm.B = B;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.Nq = Nq;
  prm.P = page_size;
  prm.max_pages = max_pages;
  prm.num_pages = num_pages;
  // the caches as [num_pages * Hkv][P][d]: one box = 64 features of the P
  // rows of one (page, kv head)
  if (static_cast<int64_t>(num_pages) * Hkv > INT32_MAX) return FA_ERR_UNSUPPORTED;
  const CUtensorMapDataType tdt = dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!make_map(&prm.tm_k, k_cache, tdt, 2, d, page_size, static_cast<uint64_t>(num_pages) * Hkv, 64, page_size) ||
      !make_map(&prm.tm_v, v_cache, tdt, 2, d, page_size, static_cast<uint64_t>(num_pages) * Hkv, 64, page_size))
    return FA_ERR_CUDA;
  prm.S = fa::decode_splits(B, Hkv, d, max_pages);
  // a split holds whole tiles of 128 keys
  const int ppt = fa::kDecodeTile / page_size;
  prm.pages_per_split = ((max_pages + prm.S - 1) / prm.S + ppt - 1) / ppt * ppt;
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  const int64_t rows = static_cast<int64_t>(B) * Hq * Nq;
  prm.part_o = static_cast<float*>(workspace);
  prm.part_ml = prm.part_o + rows * prm.S * d;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == FA_BF16;
  const int R = (Hq / Hkv) * Nq;
  const int rb = R <= 4 ? 4 : R <= 8 ? 8 : R <= 16 ? 16 : 32;
  // q as [B * Hq * Nq][d]; a box is the NP (rows padded to 16 or 32) rows
  // that start at an item's first row
  const int np = rb < 16 ? 16 : rb;
  if (!make_map(&prm.tm_q, q, tdt, 2, d, static_cast<uint64_t>(B) * Hq * Nq, 1, 64, np)) return FA_ERR_CUDA;
  const int64_t n_work = static_cast<int64_t>(B) * Hkv * prm.S;
  if (n_work > INT32_MAX) return FA_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  auto run = [&](auto split_kern, auto merge_kern, int smem) -> fa_status_t {
    fa_status_t r = opt_in_smem(split_kern, smem);
    if (r != FA_OK) return r;
    // persistent: as many blocks as fit on the GPU at once, each taking
    // work items (splits) in turn
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, split_kern, fa::kDecodeThreads, smem) !=
            cudaSuccess ||
        per_sm <= 0)
      return FA_ERR_CUDA;
    const int grid = static_cast<int>(std::min<int64_t>(n_work, static_cast<int64_t>(sms) * per_sm));
    if (launch_dependent(split_kern, static_cast<unsigned>(grid), fa::kDecodeThreads, smem, st, prm) !=
        cudaSuccess)
      return FA_ERR_CUDA;
    return launch_dependent(merge_kern, static_cast<unsigned>(rows), static_cast<unsigned>(d), 0, st, prm) ==
                   cudaSuccess
               ? FA_OK
               : FA_ERR_CUDA;
  };
#define FA_DECODE_RUN(HD, BFV, RBV)                                                                  \
  run(fa::fa_decode_split_kernel<HD, BFV, RBV>, fa::fa_decode_merge_kernel<HD, BFV>, \
      fa::DecodeLayout<HD, RBV>::kDynSmem)
#define FA_DECODE_RB(HD, BFV)                                                        \
  (rb == 4 ? FA_DECODE_RUN(HD, BFV, 4) : rb == 8 ? FA_DECODE_RUN(HD, BFV, 8)        \
             : rb == 16 ? FA_DECODE_RUN(HD, BFV, 16) : FA_DECODE_RUN(HD, BFV, 32))
  fa_status_t rs;
  if (d == 128)
    rs = bf ? FA_DECODE_RB(128, true) : FA_DECODE_RB(128, false);
  else
    rs = bf ? FA_DECODE_RB(64, true) : FA_DECODE_RB(64, false);
#undef FA_DECODE_RB
#undef FA_DECODE_RUN
  return rs;
}

}  // extern "C"

namespace {

// Checks shared by the paged-cache entry points (sizes, types, page geometry).
fa_status_t check_paged(int B, int Hq, int Hkv, int N, int d, int page_size, int max_pages, int num_pages,
                        fa_dtype_t dtype) {
  if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_pages <= 0 || num_pages <= 0)
    return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 127 ||
      static_cast<int64_t>(num_pages) * Hkv > INT32_MAX || static_cast<int64_t>(B) * Hq > INT32_MAX ||
      static_cast<int64_t>(B) * Hq * N > INT32_MAX)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// How a pass over the paged cache is cut into blocks.
struct PagedPlan {
  int toks, seqs;   // a row tile: tokens x sequences (x G heads)
  int n_tiles;      // row tiles of an owner
  int n_pairs;      // the first 2 n_pairs of them in pairs, the others one by one
  int64_t owners;   // kv heads, of every sequence in the forward pass
  int S, S_single;  // key splits of a pair of row tiles / of an odd last one
  bool joined;      // partial results go through the workspace
  int slots() const { return std::max(n_pairs ? S : 0, n_tiles > 2 * n_pairs ? S_single : 0); }
  int64_t rows() const { return owners * n_tiles * 128; }
  size_t o_bytes(int d) const { return joined ? static_cast<size_t>(rows()) * slots() * d * 4u : 0; }
  size_t bytes(int d) const { return joined ? o_bytes(d) + static_cast<size_t>(rows()) * slots() * 8u : 0; }
};

// Splits by a model of the time, in steps of one row tile on one key tile
// (1 us, half of a pair's): a block costs its steps and 5 more for its start
// and end; blocks run in whole waves of one per SM (they are about equally
// long); joining costs 5 steps for the launch and the partial results' way
// through L2 (a row of a split: 8 d + 16 bytes at 5 TB/s).  Up to a wave of
// splits, at least 2 key tiles each.
// Against the best of up to 36 other plans (each timed; 1 to 15 row tiles of 1,
// 8 and 12 kv heads on 2048 to 65 536 keys; 1 to 8 sequences of 32 to 800 new
// tokens behind 250 to 16 000) the plan is 0.2 % slower on average behind a
// prefix and 2 % in the forward pass, at worst 5 and 23 %.  With fractions of a
// wave from 4 waves on, 1.3 and 3 %, at worst 29 (15 row tiles x 8 heads on
// 65 536 keys: 704 us in 5 splits of singles, 548 in 7 of pairs) and 39 %.
PagedPlan paged_plan(int B, int Hq, int Hkv, int N, int d, int64_t keys, bool prefix) {
  PagedPlan pl;
  const int G = Hq / Hkv;
  pl.toks = prefix ? N : std::min(N, 128 / G);
  pl.seqs = prefix ? std::min(B, 128 / (G * N)) : 1;
  pl.n_tiles = static_cast<int>(prefix ? (static_cast<int64_t>(B) + pl.seqs - 1) / pl.seqs
                                       : (static_cast<int64_t>(N) + pl.toks - 1) / pl.toks);
  pl.owners = prefix ? Hkv : static_cast<int64_t>(B) * Hkv;
  if (prefix && keys == 0) {  // nothing shared: no blocks, no partial results
    pl.n_pairs = pl.S = pl.S_single = 0;
    pl.joined = true;
    return pl;
  }
  const int64_t tiles = std::max<int64_t>(1, (keys + 127) / 128);
  const int64_t cap = std::min<int64_t>(fa::kDecodeSMs, std::max<int64_t>(1, tiles / 2));
  pl.n_pairs = 0;
  pl.S = pl.S_single = 1;
  double best = 1e300;
  // Pairs read each key once for two row tiles: 3 % in favour of pairs where
  // the model puts both alike.  (8 heads on 65 536 keys, pairs against singles:
  // 2 row tiles 84.0 and 83.0 us, 3: 118.8 and 114.1, 4: 141 and 156, 6: 205 and
  // 213, 9: 306 and 331.)  Row tiles one by one only while they do not fill
  // the GPU.
  for (const int64_t pairs : {static_cast<int64_t>(pl.n_tiles / 2), static_cast<int64_t>(0)}) {
    const int64_t odd = pl.n_tiles - 2 * pairs;
    for (int64_t S = 1; S <= cap; ++S) {
      const int64_t Ss = odd ? (pairs ? (S + 1) / 2 : S) : 1;
      const int64_t blocks = pl.owners * (pairs * S + odd * Ss);
      if (S > 1 && blocks > 8 * fa::kDecodeSMs) break;  // the GPU is full
      const double waves = static_cast<double>((blocks + fa::kDecodeSMs - 1) / fa::kDecodeSMs);
      const double steps = std::max(pairs ? 2.0 * ((tiles + S - 1) / S) : 0.0, odd ? 1.0 * ((tiles + Ss - 1) / Ss) : 0.0);
      double cost = waves * (steps + 5);
      if (S > 1 || prefix) cost += 5 + static_cast<double>(pl.rows()) * S * (8.0 * d + 16) / 5e12 / 1e-6;
      if (!pairs) cost *= 1.03;
      if (cost < best) {
        best = cost;
        pl.n_pairs = static_cast<int>(pairs);
        pl.S = static_cast<int>(pairs ? S : Ss);
        pl.S_single = static_cast<int>(odd ? Ss : S);
      }
    }
    if (pl.n_tiles < 2 || pl.owners * pl.n_tiles > fa::kDecodeSMs) break;
  }
  pl.joined = prefix || pl.slots() > 1;
  return pl;
}

struct PagedArgs {
  const void *q, *k_cache, *v_cache;
  const int *table, *lens, *new_lens;
  void* o;
  float* lse;
  int B, Hq, Hkv, N, d, P, max_pages, num_pages;
  bool decode;       // behind a prefix
  int prefix;        // keys of it that the row-tile pass takes
  int shared_pages;  // pages of it that the own-key pass takes
  float scale;
  fa_dtype_t dtype;
};

// Splits of each sequence's own keys: as many as bring the blocks nearest to
// two per SM, of at least 1024 keys each.  8192 own keys, 32/8 heads of 128: 1
// sequence 83 us in one piece, 18.9 in 8; 8 sequences 84 and 49 in 4; but 28 and
// 32 sequences 142 and 162 us in one piece, 163 and 188 in two (with 2048 keys
// 40 and 46, 51 and 58).  The 1024: own_keys is what the table has room for.
// Full tables would gain from shorter splits (2048 keys of 1 sequence: 16.9 us
// in 2, 10.9 in 8), but sequences that fill little of theirs pay for each (150
// keys: 5.1 us in one piece, 7.2 in 2, 10.8 in 16).
int own_splits(int B, int Hkv, int64_t own_keys) {
  const int64_t items = static_cast<int64_t>(B) * Hkv, slots = 2 * fa::kDecodeSMs;
  return static_cast<int>(std::max<int64_t>(1, std::min((2 * slots + items) / (2 * items), own_keys / 1024)));
}

// Keys of the prefix that get a pass of their own.  A short one is read with
// the own keys of every sequence instead: one kernel, and while the blocks'
// reads of it stay few.  Both ways timed (own keys' kernel alone | pass and own
// keys) at 396 sizes: 32/8, 12/12, 16/16, 8/1 and 28/4 heads of 64 and 128, 1 to
// 32 rows, 1 to 128 sequences, 64 to 1024 keys.  32/8 x 128: 512 keys, 1 to 32
// sequences 9.8-12.7 | 12.5-15.2 us, 64: 24.2 | 21.0; 256 keys, 64: 17.6 | 20.0,
// 128: 28.1 | 27.1; 768 keys, 4: 12.8 | 13.8; 1024 keys, 4: 15.3 | 14.3.  Heads
// of 64 are read in half the time (256 keys, 128 sequences: 17.0 | 18.9).  The
// rule is 0.4 % above the better of the two on average; at most 8 % where it
// leaves the pass out (4 tokens of 1 sequence, 8/1 heads, 768 keys: 25.6 | 23.7)
// and 19 % where it does not (4 tokens of 16, 32/8, 1024: 19.1 | 22.7).
int own_pass_prefix(int B, int Hkv, int d, int prefix_len) {
  return prefix_len <= 768 && static_cast<int64_t>(B) * Hkv * prefix_len * d <= (1 << 24) ? 0 : prefix_len;
}

size_t own_bytes(int B, int Hq, int N, int d, int S) {
  return S > 1 ? static_cast<size_t>(B) * Hq * N * S * (static_cast<size_t>(d) + 2) * 4u : 0;
}

// The paged kernel, where there are keys for it (a forward pass, a long
// prefix); in decode the kernel over each sequence's own keys; the merge kernel
// where the results of several blocks are joined (the own-key kernel does that
// itself for the prefix's when its own keys are not split).
fa_status_t paged_run(const PagedArgs& a, const PagedPlan& pl, void* workspace, void* stream) {
  fa_status_t s = check_device();
  if (s != FA_OK) return s;
  const bool bf = a.dtype == FA_BF16;
  const CUtensorMapDataType dt = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int G = a.Hq / a.Hkv, d = a.d;
  fa::PagedMergeParams mp;
  std::memset(&mp, 0, sizeof(mp));
  fa::PagedParams prm;
  std::memset(&prm, 0, sizeof(prm));
  const int64_t singles = pl.n_tiles - 2 * static_cast<int64_t>(pl.n_pairs);
  const int64_t blocks = pl.owners * (static_cast<int64_t>(pl.n_pairs) * pl.S + singles * pl.S_single);
  if (blocks > INT32_MAX) return FA_ERR_UNSUPPORTED;
  if (blocks > 0) {
    auto enc = encode_fn();
    if (!enc) return FA_ERR_CUDA;
    const cuuint64_t rb = static_cast<cuuint64_t>(d) * 2;  // bytes of a row
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(G), static_cast<cuuint64_t>(a.N),
                                static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.B)};
    const cuuint64_t strides[4] = {rb * a.N, rb, rb * a.N * G, rb * a.N * a.Hq};
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(pl.toks), 1,
                               static_cast<cuuint32_t>(pl.seqs)};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    if (enc(&prm.tm_q, dt, 5, const_cast<void*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return FA_ERR_CUDA;
    const uint64_t outer = static_cast<uint64_t>(a.num_pages) * a.Hkv;
    if (!make_map(&prm.tm_k, a.k_cache, dt, 2, d, a.P, outer, 64, a.P) ||
        !make_map(&prm.tm_v, a.v_cache, dt, 2, d, a.P, outer, 64, a.P))
      return FA_ERR_CUDA;
  }
  prm.table = a.table;
  prm.lens = a.lens;
  prm.new_lens = a.new_lens;
  prm.o = a.o;
  prm.lse = a.lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (pl.joined) {
    prm.part_o = reinterpret_cast<float4*>(ws);
    prm.part_ml = reinterpret_cast<float2*>(ws + pl.o_bytes(d));
  }
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.G = G;
  prm.N = a.N;
  prm.P = a.P;
  prm.max_pages = a.max_pages;
  prm.num_pages = a.num_pages;
  prm.decode = a.decode ? 1 : 0;
  prm.prefix = a.prefix;
  prm.toks = pl.toks;
  prm.seqs = pl.seqs;
  prm.n_tiles = pl.n_tiles;
  prm.n_pairs = pl.n_pairs;
  prm.S = pl.S;
  prm.S_single = pl.S_single;
  prm.slots = pl.slots();
  prm.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  auto run = [&](auto kern, auto own1, auto own2, auto merge, int smem) -> fa_status_t {
    fa_status_t r = FA_OK;
    if (blocks > 0) {
      if ((r = opt_in_smem(kern, smem)) != FA_OK) return r;
      if (launch_dependent(kern, dim3(static_cast<unsigned>(blocks)), fa::kFwdThreads, smem, st, prm) != cudaSuccess)
        return FA_ERR_CUDA;
    }
    if (a.decode) {
      fa::OwnParams op;
      std::memset(&op, 0, sizeof(op));
      op.p = prm;
      op.S = own_splits(a.B, a.Hkv, static_cast<int64_t>(a.max_pages) * a.P - a.prefix);
      const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * op.S;
      if (items > INT32_MAX) return FA_ERR_UNSUPPORTED;
      if (op.S > 1) {
        op.own_o = reinterpret_cast<float*>(ws + pl.bytes(d));
        op.own_ml = op.own_o + static_cast<size_t>(a.B) * a.Hq * a.N * op.S * d;
      }
      op.shared_pages = a.shared_pages;
      while ((1 << op.log2P) < a.P) ++op.log2P;
      op.q = a.q;
      op.k_cache = a.k_cache;
      op.v_cache = a.v_cache;
      // rings as deep as the blocks that share an SM allow
      const int slots = op.S == 1 ? pl.slots() : 0;
      const int per_sm = static_cast<int>(
          std::min<int64_t>(fa::own_blocks_per_sm(d), (items + fa::kDecodeSMs - 1) / fa::kDecodeSMs));
      op.stages = fa::kOwnMaxStages;
      while (op.stages > 2 && (fa::own_smem(d, op.stages, G * a.N, slots) + 1024) * per_sm > 228 * 1024) --op.stages;
      const int own_smem = fa::own_smem(d, op.stages, G * a.N, slots);
      auto own = G * a.N > 16 ? own2 : own1;
      if ((r = opt_in_smem(own, fa::kOwnSmemLimit)) != FA_OK) return r;
      if (launch_dependent(own, dim3(static_cast<unsigned>(items)), fa::kOwnThreads, own_smem, st, op) != cudaSuccess)
        return FA_ERR_CUDA;
      if (op.S == 1) return FA_OK;
      mp.own_o = op.own_o;
      mp.own_ml = op.own_ml;
      mp.own_S = op.S;
    } else if (!pl.joined) {
      return FA_OK;
    }
    mp.p = prm;
    const int64_t grid = pl.rows() / (1024 / d);
    return launch_dependent(merge, dim3(static_cast<unsigned>(grid)), 256, 0, st, mp) == cudaSuccess ? FA_OK
                                                                                                   : FA_ERR_CUDA;
  };
#define FA_PAGED_RUN(HD, BFV) \
  run(fa::fa_paged_kernel<HD, BFV>, fa::fa_prefix_own_kernel<HD, BFV, 1>, fa::fa_prefix_own_kernel<HD, BFV, 2>, \
      fa::fa_paged_merge_kernel<HD, BFV>, fa::PagedLayout<HD>::kBytes)
  if (d == 128) return bf ? FA_PAGED_RUN(128, true) : FA_PAGED_RUN(128, false);
  return bf ? FA_PAGED_RUN(64, true) : FA_PAGED_RUN(64, false);
#undef FA_PAGED_RUN
}

}  // namespace

extern "C" {

fa_status_t fa_append_paged(const void* q, const void* k, const void* v, const int64_t* strides, void* q_out,
                            void* k_out, void* k_cache, void* v_cache, const int* block_table,
                            const int* seq_lens, const int* new_lens, const float* inv_freq, int B, int Hq,
                            int Hkv, int N, int d, int page_size, int max_pages, int num_pages, int rot_dim,
                            int interleaved, fa_dtype_t dtype, void* stream) {
  fa_status_t s = check_paged(B, Hq, Hkv, N, d, page_size, max_pages, num_pages, dtype);
  if (s != FA_OK) return s;
  if (rot_dim < 0 || rot_dim > d || (interleaved != 0 && interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return FA_OK;
  if (!k || !v || !k_cache || !v_cache || !block_table || !seq_lens || (q == nullptr) != (q_out == nullptr) ||
      (rot_dim > 0 && !inv_freq))
    return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(new_lens) || !aligned4(inv_freq))
    return FA_ERR_MISALIGNED;
  fa::AppendParams prm;
  std::memset(&prm, 0, sizeof(prm));
  for (int i = 0; i < 3; ++i) {
    const int64_t heads = i == 0 ? Hq : Hkv;
    const int64_t dense[3] = {heads * N * d, static_cast<int64_t>(N) * d, d};
    const int64_t extent[3] = {B, heads, N};  // a dimension of one entry is never stepped over
    long long* dst = i == 0 ? prm.qs : i == 1 ? prm.ks : prm.vs;
    for (int j = 0; j < 3; ++j) {
      dst[j] = extent[j] == 1 ? 0 : strides ? strides[3 * i + j] : dense[j];
      if (dst[j] % 8 != 0 && (i > 0 || q)) return FA_ERR_MISALIGNED;  // rows start on 16-byte boundaries
    }
  }
  if ((s = check_device()) != FA_OK) return s;
  prm.q = q;
  prm.k = k;
  prm.v = v;
  prm.q_out = q_out;
  prm.k_out = k_out;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.table = block_table;
  prm.lens = seq_lens;
  prm.new_lens = new_lens;
  prm.inv_freq = inv_freq;
  prm.tokens = static_cast<long long>(B) * N;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.N = N;
  prm.d = d;
  prm.P = page_size;
  prm.max_pages = max_pages;
  prm.num_pages = num_pages;
  prm.rot = rot_dim;
  // tokens of a block: as many as its threads hold (one head lane), fewer
  // when there are few tokens, so that the heads spread over the threads
  const int rows = fa::kAppendThreads / (d / 16);
  int tpb = 1;
  while (tpb < rows && tpb < prm.tokens) tpb *= 2;
  prm.tok_per_block = tpb;
  const int64_t gx = (prm.tokens + tpb - 1) / tpb;
  if (gx > INT32_MAX) return FA_ERR_UNSUPPORTED;
  // The heads in gy parts: enough blocks for kBlocks per SM as long as threads
  // keep whole rounds of kAppendHeads heads, and for one per SM as long as
  // they keep a head.
  constexpr int64_t kBlocks = 24;
  const int heads = (q ? Hq : 0) + 2 * Hkv, lanes = rows / tpb;
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const int64_t most = (heads + lanes - 1) / lanes;  // heads of a thread with gy = 1
  auto parts = [&](int64_t per_sm) { return (per_sm * sms + gx - 1) / gx; };
  const int64_t rounds = std::max<int64_t>(1, most / (fa::kAppendHeads * parts(kBlocks)));
  const int64_t whole = std::max<int64_t>(1, most / (fa::kAppendHeads * rounds));
  const int64_t gy = std::min<int64_t>(std::max(std::min(whole, parts(kBlocks)), std::min(most, parts(1))), 65535);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == FA_BF16;
  auto kern = bf ? (interleaved ? fa::fa_append_kernel<true, true> : fa::fa_append_kernel<true, false>)
                 : (interleaved ? fa::fa_append_kernel<false, true> : fa::fa_append_kernel<false, false>);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  return launch_dependent(kern, grid, fa::kAppendThreads, 0, st, prm) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fwd_paged_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int page_size, int max_pages) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || d <= 0 || page_size <= 0 || max_pages <= 0 || Hq % Hkv != 0 ||
      Hq / Hkv > 128)
    return 0;
  return paged_plan(B, Hq, Hkv, N, d, static_cast<int64_t>(max_pages) * page_size, false).bytes(d);
}

fa_status_t fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                         const int* seq_lens, const int* new_lens, void* o, float* lse, int B, int Hq, int Hkv,
                         int N, int d, int page_size, int max_pages, int num_pages, float scale,
                         fa_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status_t s = check_paged(B, Hq, Hkv, N, d, page_size, max_pages, num_pages, dtype);
  if (s != FA_OK) return s;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o || !lse) return FA_ERR_INVALID_ARG;
  const PagedPlan pl = paged_plan(B, Hq, Hkv, N, d, static_cast<int64_t>(max_pages) * page_size, false);
  if (pl.bytes(d) > 0 && (!workspace || workspace_bytes < pl.bytes(d))) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(workspace) ||
      !aligned4(lse) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned4(new_lens))
    return FA_ERR_MISALIGNED;
  return paged_run({q, k_cache, v_cache, block_table, seq_lens, new_lens, o, lse, B, Hq, Hkv, N, d, page_size,
                    max_pages, num_pages, false, 0, 0, scale, dtype},
                   pl, workspace, stream);
}

size_t fa_decode_prefix_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int page_size, int max_pages,
                                        int prefix_len) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || d <= 0 || page_size <= 0 || max_pages <= 0 || prefix_len < 0 ||
      Hq % Hkv != 0 || static_cast<int64_t>(Hq / Hkv) * Nq > fa::kDecodeMaxRows)
    return 0;
  const int pass = own_pass_prefix(B, Hkv, d, prefix_len);
  return paged_plan(B, Hq, Hkv, Nq, d, pass, true).bytes(d) +
         own_bytes(B, Hq, Nq, d, own_splits(B, Hkv, static_cast<int64_t>(max_pages) * page_size - pass));
}

fa_status_t fa_decode_prefix(const void* q, const void* k_cache, const void* v_cache, const int* block_table,
                             const int* seq_lens, void* o, float* lse, int B, int Hq, int Hkv, int Nq, int d,
                             int page_size, int max_pages, int num_pages, int prefix_len, float scale,
                             fa_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status_t s = check_paged(B, Hq, Hkv, Nq, d, page_size, max_pages, num_pages, dtype);
  if (s != FA_OK) return s;
  if (Nq <= 0 || !std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (prefix_len < 0 || prefix_len > max_pages * page_size || prefix_len % page_size != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(Hq / Hkv) * Nq > fa::kDecodeMaxRows) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !o || !lse) return FA_ERR_INVALID_ARG;
  const int pass = own_pass_prefix(B, Hkv, d, prefix_len);
  const PagedPlan pl = paged_plan(B, Hq, Hkv, Nq, d, pass, true);
  const size_t need = pl.bytes(d) + own_bytes(B, Hq, Nq, d,
                                              own_splits(B, Hkv, static_cast<int64_t>(max_pages) * page_size - pass));
  if (need > 0 && (!workspace || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(workspace) ||
      !aligned4(lse) || !aligned4(block_table) || !aligned4(seq_lens))
    return FA_ERR_MISALIGNED;
  return paged_run({q, k_cache, v_cache, block_table, seq_lens, nullptr, o, lse, B, Hq, Hkv, Nq, d, page_size,
                    max_pages, num_pages, true, pass, pass == 0 ? prefix_len / page_size : 0, scale, dtype},
                   pl, workspace, stream);
}

fa_status_t fa_set_bwd_max_blocks(int max_blocks) {
  if (max_blocks < 0) return FA_ERR_INVALID_ARG;
  g_bwd_max_blocks.store(max_blocks);
  return FA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Fixed scratch for fa_bwd_noalloc: reserved in the device memory of every GPU
// that loads this library, for the life of the process.  Host code must not
// pass `g_bwd_noalloc_scratch` itself to a kernel (on the host the name is
// only a stand-in); its device address is looked up once per device with
// cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_bwd_noalloc_scratch[FA_BWD_NOALLOC_SCRATCH_BYTES];

namespace {
std::mutex g_noalloc_mu;
void* g_noalloc_ptr[64] = {nullptr};

// Device address of the scratch array on the current device (looked up on
// the first call per device).
fa_status_t noalloc_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev < 0 || dev >= 64) return FA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_bwd_noalloc_scratch) != cudaSuccess || p == nullptr)
      return FA_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return FA_OK;
}
}  // namespace

extern "C" {

fa_status_t fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, void* dq, void* dk, void* dv,
                           int B, int Hq, int Hkv, int N, int d, float scale, int causal,
                           fa_dtype_t dtype, void* stream) {
  bool empty = false;
  fa_status_t s = check_common(B, Hq, Hkv, N, d, scale, causal, dtype, &empty);
  if (s != FA_OK) return s;
  if (empty) return FA_OK;
  const size_t need = fa::bwd_workspace_bytes(B, Hq, N, d);
  if (need > FA_BWD_NOALLOC_SCRATCH_BYTES) return FA_ERR_UNSUPPORTED;
  if ((s = check_device()) != FA_OK) return s;
  void* scratch = nullptr;
  if ((s = noalloc_scratch(&scratch)) != FA_OK) return s;
  return fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, scale, causal, dtype,
                scratch, FA_BWD_NOALLOC_SCRATCH_BYTES, stream);
}

const char* fa_status_string(fa_status_t status) {
  switch (status) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration or device";
    case FA_ERR_MISALIGNED: return "tensor pointer not 16-byte aligned";
    case FA_ERR_CUDA: return "CUDA error";
    case FA_ERR_TIMEOUT: return "device-side barrier wait timed out";
  }
  return "unknown status";
}

}  // extern "C"
