// coda.cu -- libcoda.so: kernels of the GEMM -> residual -> RMSNorm -> GEMM chain
// and the C ABI declared in include/coda.h.
//
// Forward (CODA blog, blog.hotdry.top, section
// "GEMM-Residual-RMSNorm-GEMM 重参数化", its three steps):
//   launch 1  GEMM0 x @ W0 with EpiResidualGammaSumsq   -> h, hg = h*gamma, partial sum h^2
//   launch 2  rowreduce_rsqrt_kernel                    -> r = 1/sqrt(sum/d + eps)
//   launch 3  GEMM1 hg @ W1 with EpiRowScale            -> y = r * acc
// Backward data gradient (section "反向传播的 GEMM-Epilogue 结构"):
//   launch 1  GEMM dy @ W1^T with EpiRmsNormBackward    -> grad_h (cooperative launch)

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <random>
#include <tuple>
#include <vector>

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "coda.h"
#include "attn_q8.cuh"
#include "attn_q8_tile.cuh"
#include "cache_q8.cuh"
#include "epilogues.cuh"
#include "gemm_pair.cuh"
#include "q8.cuh"
#include "q8_mid.cuh"
#include "q8_small.cuh"

namespace coda {

// ---------------------------------------------------------------------------
// auxiliary kernels
// ---------------------------------------------------------------------------

// Step 2 of the forward: the light auxiliary reduction over the per-tile
// partial sums of squares (fixed summation order over tiles).
__global__ void rowreduce_rsqrt_kernel(const float* __restrict__ part, int nt, int M, int d,
                                       float eps, float* __restrict__ r) {
  griddep_launch_dependents();
  griddep_wait();
  const int m = blockIdx.x * blockDim.x + threadIdx.x;
  if (m >= M) return;
  float s = 0.f;
  for (int t = 0; t < nt; ++t) s += __ldg(part + static_cast<size_t>(t) * M + m);
  r[m] = rsqrtf(s / static_cast<float>(d) + eps);
}

// Auxiliary reduction of the backward statistic: s[m] = sum_t spart[t][m]
// (fixed summation order over tiles).
__global__ void rowsum_kernel(const float* __restrict__ part, int nt, int M, float* __restrict__ s) {
  griddep_launch_dependents();
  griddep_wait();
  const int m = blockIdx.x * blockDim.x + threadIdx.x;
  if (m >= M) return;
  float acc = 0.f;
  for (int t = 0; t < nt; ++t) acc += __ldg(part + static_cast<size_t>(t) * M + m);
  s[m] = acc;
}

// dgamma[j] = sum_i gpart[i][j] over the per-warp column partials (fixed order).
__global__ void colsum_kernel(const float* __restrict__ part, int nrows, int d,
                              float* __restrict__ out) {
  griddep_launch_dependents();
  griddep_wait();
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= d) return;
  float acc = 0.f;
  for (int i = 0; i < nrows; ++i) acc += __ldg(part + static_cast<size_t>(i) * d + j);
  out[j] = acc;
}

// Standalone RMSNorm of the unfused reference sequence: reads h, writes
// hn = bf16(r * h * gamma) and r.  One block of 256 threads per row.
__global__ void __launch_bounds__(256) rmsnorm_rows_kernel(const __nv_bfloat16* __restrict__ h,
                                                           const __nv_bfloat16* __restrict__ gamma,
                                                           float eps, int M, int d,
                                                           __nv_bfloat16* __restrict__ hn,
                                                           float* __restrict__ r) {
  __shared__ float warp_sums[8];
  griddep_launch_dependents();
  griddep_wait();
  const int m = blockIdx.x;
  if (m >= M) return;
  const __nv_bfloat16* row = h + static_cast<size_t>(m) * d;
  const int nchunks = d / 8;
  float ss = 0.f;
  for (int i = threadIdx.x; i < nchunks; i += blockDim.x) {
    const Chunk8 c = ldg8(row + 8 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf16lo(c.w[e]), b = bf16hi(c.w[e]);
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = ss;
  __syncthreads();
  float tot = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) tot += warp_sums[w];
  const float rr = rsqrtf(tot / static_cast<float>(d) + eps);
  if (threadIdx.x == 0) r[m] = rr;
  __nv_bfloat16* out = hn + static_cast<size_t>(m) * d;
  for (int i = threadIdx.x; i < nchunks; i += blockDim.x) {
    const Chunk8 c = ldg8(row + 8 * i);
    const Chunk8 g = ldg8(gamma + 8 * i);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(rr * bf16lo(c.w[e]) * bf16lo(g.w[e]), rr * bf16hi(c.w[e]) * bf16hi(g.w[e]));
    stg8(out + 8 * i, w);
  }
}

__device__ uint64_t g_selftest_flag = 0;  // never written by anyone

// Watchdog self-test: both waits run out by construction.
__global__ void watchdog_selftest_kernel(uint64_t timeout_ns) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ __align__(8) uint64_t bar;
  __shared__ uint32_t abort_flag;
  if (threadIdx.x != 0) return;
  abort_flag = 0u;
  const uint32_t b = smem_u32(&bar);
  mbar_init(b, 1);
  fence_mbar_init();
  WaitCtl wc{timeout_ns, &g_coda_status, &abort_flag};
  bounded_wait(b, 0u, wc, kSiteSelftestBarrier);  // nobody arrives
  flag_wait(&g_selftest_flag, 1ull, wc, kSiteSelftestFlag);  // nobody sets it
}

static auto* const kGemm0 = &gemm_epilogue_kernel<EpiResidualGammaSumsq, true>;
static auto* const kGemm1 = &gemm_epilogue_kernel<EpiRowScale, true>;
static auto* const kDgrad = &gemm_epilogue_kernel<EpiRmsNormBackward, false>;
static auto* const kPairGemm0 = &gemm_pair_epilogue_kernel<EpiResidualGammaSumsq, true>;
static auto* const kPairGemm1 = &gemm_pair_epilogue_kernel<EpiRowScale, true>;
static auto* const kPairDgrad = &gemm_pair_epilogue_kernel<EpiRmsNormBackward, false>;
static auto* const kDgradFull = &gemm_epilogue_kernel<EpiRmsNormBackwardFull, false>;
static auto* const kPairDgradFull = &gemm_pair_epilogue_kernel<EpiRmsNormBackwardFull, false>;
static auto* const kGemm1Swiglu = &gemm_epilogue_kernel<EpiRowScaleSwiGLU, true>;
static auto* const kPairGemm1Swiglu = &gemm_pair_epilogue_kernel<EpiRowScaleSwiGLU, true>;
static auto* const kSwigluBwd = &gemm_epilogue_kernel<EpiSwiGLUBackward, false>;
static auto* const kWgrad = &gemm_epilogue_kernel<EpiStoreF32, true, true>;
static auto* const kPairGemm0F8 = &gemm_pair_epilogue_kernel<EpiResidualGammaSumsqFp8, true, false, true>;
static auto* const kPairGemm1F8 = &gemm_pair_epilogue_kernel<EpiRowScaleFp8, true, false, true>;
static auto* const kPairWgrad = &gemm_pair_epilogue_kernel<EpiStoreF32, true, true>;
static auto* const kXgrad = &gemm_epilogue_kernel<EpiRowScale, false>;
static auto* const kPairXgrad = &gemm_pair_epilogue_kernel<EpiRowScale, false>;
static auto* const kPairSwigluBwd = &gemm_pair_epilogue_kernel<EpiSwiGLUBackward, false>;
static auto* const kSwigluBwdQ8 = &gemm_epilogue_kernel<EpiSwiGLUBackwardQ8, false>;
static auto* const kPairSwigluBwdQ8 = &gemm_pair_epilogue_kernel<EpiSwiGLUBackwardQ8, false>;
static auto* const kProductQ8 = &gemm_epilogue_kernel<EpiTokenChannelScale, true>;
static auto* const kPairProductQ8 = &gemm_pair_epilogue_kernel<EpiTokenChannelScale, true>;
static auto* const kProductSmall1 = &product_q8_small_kernel<1>;  // groups of 8 tokens
static auto* const kProductSmall2 = &product_q8_small_kernel<2>;
static auto* const kProductSmall4 = &product_q8_small_kernel<4>;
static auto* const kProductMid = &product_q8_mid_kernel<false>;
static auto* const kProductNarrow = &product_q8_mid_kernel<true>;
static auto* const kDgradGivenS = &gemm_epilogue_kernel<EpiRmsNormBackwardGivenS, false>;
static auto* const kPairDgradGivenS = &gemm_pair_epilogue_kernel<EpiRmsNormBackwardGivenS, false>;

// dynamic shared memory of each kernel (ring, barriers, the policy's staging buffers)
constexpr uint32_t kGemm0Smem = cta_smem_bytes<EpiResidualGammaSumsq>();
constexpr uint32_t kGemm1Smem = cta_smem_bytes<EpiRowScale>();
constexpr uint32_t kDgradSmem = cta_smem_bytes<EpiRmsNormBackward>();
constexpr uint32_t kPairGemm0Smem = pair_smem_bytes<EpiResidualGammaSumsq>();
constexpr uint32_t kPairGemm1Smem = pair_smem_bytes<EpiRowScale>();
constexpr uint32_t kPairDgradSmem = pair_smem_bytes<EpiRmsNormBackward>();
constexpr uint32_t kDgradFullSmem = cta_smem_bytes<EpiRmsNormBackwardFull>();
constexpr uint32_t kPairDgradFullSmem = pair_smem_bytes<EpiRmsNormBackwardFull>();
constexpr uint32_t kGemm1SwigluSmem = cta_smem_bytes<EpiRowScaleSwiGLU>();
constexpr uint32_t kPairGemm1SwigluSmem = pair_smem_bytes<EpiRowScaleSwiGLU>();
constexpr uint32_t kSwigluBwdSmem = cta_smem_bytes<EpiSwiGLUBackward>();
constexpr uint32_t kWgradSmem = cta_smem_bytes<EpiStoreF32>();
constexpr uint32_t kPairGemm0F8Smem = pair_smem_bytes<EpiResidualGammaSumsqFp8>();
constexpr uint32_t kPairGemm1F8Smem = pair_smem_bytes<EpiRowScaleFp8>();
constexpr uint32_t kPairWgradSmem = pair_smem_bytes<EpiStoreF32>();
constexpr uint32_t kXgradSmem = cta_smem_bytes<EpiRowScale>();
constexpr uint32_t kPairXgradSmem = pair_smem_bytes<EpiRowScale>();
constexpr uint32_t kPairSwigluBwdSmem = pair_smem_bytes<EpiSwiGLUBackward>();
constexpr uint32_t kSwigluBwdQ8Smem = cta_smem_bytes<EpiSwiGLUBackwardQ8>();
constexpr uint32_t kPairSwigluBwdQ8Smem = pair_smem_bytes<EpiSwiGLUBackwardQ8>();
constexpr uint32_t kProductQ8Smem = cta_smem_bytes<EpiTokenChannelScale>();
constexpr uint32_t kPairProductQ8Smem = pair_smem_bytes<EpiTokenChannelScale>();
constexpr uint32_t kDgradGivenSSmem = cta_smem_bytes<EpiRmsNormBackwardGivenS>();
constexpr uint32_t kPairDgradGivenSSmem = pair_smem_bytes<EpiRmsNormBackwardGivenS>();

}  // namespace coda

// ---------------------------------------------------------------------------
// Data gradient without any allocation: scratch in a static device array.
//
// Some callers cannot call cudaMalloc (or any allocating routine) at the
// point where they run the backward: code inside a custom allocator or
// memory-pool callback, runtimes that forbid allocation while a step is in
// flight because it could synchronise the device or fragment a pre-sized
// pool, and embedders whose device memory is fully reserved up front.  For
// them this entry point takes only inputs and outputs; the partial row
// statistics and completion flags that coda_bwd_dgrad keeps in the caller's
// workspace live instead in the fixed array below, which every GPU that
// loads this library holds until the process exits.
// ---------------------------------------------------------------------------
constexpr size_t kNoAllocPartials = 2 * CODA_NOALLOC_MAX_PARTIALS;  // fp32, two per (row, column tile)
constexpr size_t kNoAllocFlags = CODA_NOALLOC_MAX_TILES;        // u64 per output tile
constexpr size_t kNoAllocFlagOffset = kNoAllocPartials * sizeof(float);
constexpr size_t kNoAllocEpochOffset = kNoAllocFlagOffset + kNoAllocFlags * sizeof(uint64_t);
constexpr size_t kNoAllocBytes = kNoAllocEpochOffset + 256;

// 4 MiB of partials + 128 KiB of flags + a 256-byte slot with the launch
// counter and its arrival word.  The flags need no clearing: each launch
// publishes counter + 1 and its last block to finish advances the counter, so
// values left by an earlier call never match (the array starts zeroed).
static __device__ __align__(256) unsigned char g_noalloc_dgrad_scratch[kNoAllocBytes];

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

using namespace coda;

constexpr int kMaxDevices = 64;
constexpr int kGroupM = 16;     // 128-row blocks per L2 group (single-CTA tiles)
constexpr int kPairGroupM = 8;  // 256-row blocks per L2 group (CTA-pair tiles)

constexpr int kRingSmem = 220 * 1024;  // of an SM, for the rings of its blocks

struct DevState {
  bool init = false;
  coda_status_t status = CODA_OK;
  int sms = 0;
  int max_pairs = 0;  // co-resident clusters of two for the CTA-pair kernels
  void* noalloc_scratch = nullptr;  // device address of g_noalloc_dgrad_scratch on this device
  int mid_clusters[2][3] = {};  // co-resident clusters of 2, 4, 8 of the mid-size product; narrow
};

std::mutex g_mu;
DevState g_dev[kMaxDevices];
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::atomic<uint64_t> g_timeout_ns{1000000000ull};
std::atomic<int> g_fold_rowreduce{0};  // 1: r computed in GEMM1's epilogue (no separate launch)
std::atomic<int> g_split_tail{1};      // 1: split tails in the CTA-pair GEMMs that qualify
std::atomic<int> g_mma_mode{1};  // 0: single-CTA 128x256 tiles, 1: CTA-pair 256x256 tiles (default)
cudaEvent_t* g_launch_events = nullptr;  // measurement hook (coda_set_launch_events)
int g_launch_events_n = 0;

// Records the measurement-hook event that follows launch k, if one is set.
void after_launch(int k, cudaStream_t stream) {
  if (g_launch_events != nullptr && k < g_launch_events_n) cudaEventRecord(g_launch_events[k], stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Every workspace starts with the 256-byte slot of the launch counter that the
// completion flags' tokens come from (launch_exit in ptx.cuh); no layout puts
// data there, so calls of any shape and entry point may share one buffer.
constexpr size_t kSlotBytes = 256;

// A fresh random 64-bit value per call, mixed into its completion flags: the
// SplitMix64 output function (Steele, Lea and Flood, "Fast splittable
// pseudorandom number generators", OOPSLA 2014) applied to a per-process seed
// plus a counter.
uint64_t next_salt() {
  static const uint64_t seed = [] {
    uint64_t v = static_cast<uint64_t>(
        std::chrono::steady_clock::now().time_since_epoch().count());
    v ^= reinterpret_cast<uintptr_t>(&v);  // differs between processes under ASLR
    try {
      std::random_device rd;
      v ^= (static_cast<uint64_t>(rd()) << 32) ^ rd();
    } catch (...) {
      // no entropy source: the clock and the address above still differ per process
    }
    return v;
  }();
  static std::atomic<uint64_t> counter{0};
  uint64_t z = seed + 0x9E3779B97F4A7C15ull * (counter.fetch_add(1) + 1);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// First use of the library on the current device (once per device, under a
// lock): checks the device, sets the kernels' shared-memory limits (which loads
// the library's device code on this device, the static scratch array of the
// no-allocation entry point included) and looks up the device address of that
// array, so that whichever entry point runs first on a device does both.
coda_status_t device_setup(int* sms, int* max_pairs = nullptr, void** noalloc_scratch = nullptr,
                           const int (**mid_clusters)[3] = nullptr) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return CODA_ERR_NO_DEVICE;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  DevState& s = g_dev[dev];
  if (!s.init) {
    int major = 0, minor = 0, count = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return CODA_ERR_NO_DEVICE;
    }
    s.sms = count;
    s.status = CODA_OK;
    if (major != 10 || minor != 3) {
      s.status = CODA_ERR_UNSUPPORTED_DEVICE;
    } else {
      bool ok = true;
      ok &= cudaFuncSetAttribute(kGemm0, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kGemm0Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kGemm1, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kGemm1Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kDgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kDgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairGemm0, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairGemm0Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairGemm1, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairGemm1Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairDgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairDgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kDgradFull, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kDgradFullSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairDgradFull, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairDgradFullSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kGemm1Swiglu, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kGemm1SwigluSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairGemm1Swiglu, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairGemm1SwigluSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kSwigluBwd, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSwigluBwdSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kWgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kWgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairGemm0F8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairGemm0F8Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairGemm1F8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairGemm1F8Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairWgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairWgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kXgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kXgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairXgrad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairXgradSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairSwigluBwd, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairSwigluBwdSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kSwigluBwdQ8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSwigluBwdQ8Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairSwigluBwdQ8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairSwigluBwdQ8Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductQ8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kProductQ8Smem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairProductQ8, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairProductQ8Smem) == cudaSuccess;
      for (auto* ring : {&row_q8_ring_kernel<false, false, false>, &row_q8_ring_kernel<true, false, false>,
                         &row_q8_ring_kernel<true, false, true>, &row_q8_ring_kernel<true, true, false>,
                         &row_q8_ring_kernel<true, true, true>})
        ok &= cudaFuncSetAttribute(ring, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem) ==
              cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductSmall1, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SmallSmem<1>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductSmall2, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SmallSmem<2>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductSmall4, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SmallSmem<4>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductMid, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 MidShape<false>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kProductNarrow, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 MidShape<true>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_tile_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 TileSmem<64>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_tile_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 TileSmem<128>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_few_kernel<64, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FewSmem<64, 1>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_few_kernel<64, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FewSmem<64, 2>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_few_kernel<128, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FewSmem<128, 1>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(&attn_q8_few_kernel<128, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FewSmem<128, 2>::kBytes) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kDgradGivenS, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kDgradGivenSSmem) == cudaSuccess;
      ok &= cudaFuncSetAttribute(kPairDgradGivenS, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairDgradGivenSSmem) == cudaSuccess;
      if (ok) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (count / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kPairDgradSmem;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kPairDgrad, &cfg) == cudaSuccess)
          s.max_pairs = std::min(clusters, count / 2);
        else
          ok = false;
      }
      for (int i = 0; ok && i < 3; ++i) {  // a cluster stays in one GPC: fewer than the SMs hold
        cudaLaunchAttribute attr = {};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2u << i;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(count) >> (i + 1) << (i + 1));
        cfg.blockDim = dim3(mid_threads(false));
        cfg.dynamicSmemBytes = MidShape<false>::kBytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        // none, for a size that does not fit (part of a device): that split is not planned
        if (cudaOccupancyMaxActiveClusters(&n, kProductMid, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        s.mid_clusters[0][i] = n;
        // Two narrow blocks share an SM (112 pairs of 32 tokens ran in one wave, 30 us, where one
        // block per SM takes two, 39 us); the occupancy query, which knows no tensor memory,
        // answers one.
        s.mid_clusters[1][i] = 2 * n;
      }
      if (g_encode == nullptr) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess && fn != nullptr) {
          g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        } else {
          ok = false;
        }
      }
      if (ok) {
        // In host code the array's name is only a host-side stand-in: its device
        // address on this device comes from the runtime.
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_dgrad_scratch) == cudaSuccess && p != nullptr)
          s.noalloc_scratch = p;
        else
          ok = false;
      }
      if (!ok) {
        cudaGetLastError();
        s.status = CODA_ERR_LAUNCH;
      }
    }
    s.init = true;
  }
  *sms = s.sms;
  if (max_pairs) *max_pairs = s.max_pairs;
  if (noalloc_scratch) *noalloc_scratch = s.noalloc_scratch;
  if (mid_clusters) *mid_clusters = s.mid_clusters;  // fixed once set
  return s.status;
}

// 2-D bf16 tensor map over a row-major [outer, inner] matrix, 128-byte swizzle.
bool tmap_2d(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_inner,
             uint32_t box_outer) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {inner * 2};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D tensor map over a row-major [outer, inner] matrix of 1-byte (FP8, INT8) codes,
// 128-byte swizzle by default.
bool tmap_2d_u8(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t outer,
                uint32_t box_inner, uint32_t box_outer,
                CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {inner};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... ExpT, typename... ActT>
cudaError_t launch_cluster(void (*kernel)(ExpT...), dim3 grid, int block, size_t smem,
                           cudaStream_t stream, bool cooperative, int cluster, ActT&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  // programmatic dependent launch for every kernel (griddep_wait in ptx.cuh)
  cudaLaunchAttribute attr[3];
  int na = 0;
  attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[na].val.programmaticStreamSerializationAllowed = 1;
  ++na;
  if (cooperative) {
    attr[na].id = cudaLaunchAttributeCooperative;
    attr[na].val.cooperative = 1;
    ++na;
  }
  if (cluster > 1) {  // blocks per cluster, for the kernels that do not fix it themselves
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = cluster;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<ActT>(args)...);
}

template <typename... ExpT, typename... ActT>
cudaError_t launch(void (*kernel)(ExpT...), dim3 grid, int block, size_t smem, cudaStream_t stream,
                   bool cooperative, ActT&&... args) {
  return launch_cluster(kernel, grid, block, smem, stream, cooperative, 1,
                        std::forward<ActT>(args)...);
}

coda_status_t check_common(int64_t M, int64_t d, int64_t N1) {
  if (M < 0 || d <= 0 || N1 <= 0) return CODA_ERR_INVALID_ARG;
  if (d % 8 != 0 || N1 % 8 != 0) return CODA_ERR_UNSUPPORTED_SHAPE;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if (M > lim || d > lim || N1 > lim) return CODA_ERR_UNSUPPORTED_SHAPE;
  return CODA_OK;
}

// ---------------------------------------------------------------------------
// Split-tail (stream-K) region of a workspace: partial accumulators, their
// flags and the launch counter that the flags' tokens come from.
// ---------------------------------------------------------------------------
constexpr int kSkMaxPairs = 80;  // no split tail for launches of more CTA pairs

// Partial slots for launches of up to `tiles` CTA-pair tiles: a split tail
// covers U + R <= 2 U - 1 tiles.
int64_t sk_slots(int64_t tiles) { return std::min<int64_t>(tiles, 2 * kSkMaxPairs); }

size_t sk_region_bytes(int64_t tiles) {
  const int64_t slots = sk_slots(tiles);
  return align256(static_cast<size_t>(slots) * 2 * kSkSlotFloats * 4) +
         align256(static_cast<size_t>(slots) * 2 * 8);
}

struct SkRegion {
  float* part = nullptr;
  uint64_t* flags = nullptr;
  uint64_t* epoch = nullptr;
  int64_t slots = 0;
};

// `slot`: the workspace's launch-counter slot (its first 256 bytes).
SkRegion sk_region(void* base, int64_t tiles, void* slot) {
  SkRegion r;
  r.slots = sk_slots(tiles);
  char* p = static_cast<char*>(base);
  r.part = reinterpret_cast<float*>(p);
  p += align256(static_cast<size_t>(r.slots) * 2 * kSkSlotFloats * 4);
  r.flags = reinterpret_cast<uint64_t*>(p);
  r.epoch = static_cast<uint64_t*>(slot);
  return r;
}

// Whole tiles for the first W - 1 waves, the last U + R tiles split along K
// (gemm_pair.cuh).  The split costs a cooperative launch (measured at 2-4 us
// when it still ended with a grid barrier) and, per pair, a partial written or
// added and sometimes a wait for
// a TMEM buffer; it gains the idle share of the last wave, (U - R) / U of a
// tile.  Measured on GB300 it pays for the llama7b and llama70b GEMM1 (R/U =
// 0.16, 64 and 128 k-blocks per tile) and loses when the last wave is mostly
// full (GEMM0 there, R/U = 0.74) or tiles are short (llama1b, 32 k-blocks).  So:
// split only when R <= U / 2 and a tile has at least 64 k-blocks, with at
// least two waves and enough slots.
SkParams plan_split_tail(const SkRegion& reg, int64_t num_tiles, int npairs, int64_t nk,
                         uint64_t salt) {
  SkParams sk = kNoSplitTail;
  if (g_split_tail.load() == 0 || reg.part == nullptr || npairs < 1 || npairs > kSkMaxPairs)
    return sk;
  const int64_t W = num_tiles / npairs, R = num_tiles % npairs;
  if (W < 2 || R == 0 || 2 * R > npairs || nk < 64 || npairs + R > reg.slots) return sk;
  sk.dp_tiles = static_cast<int>(num_tiles - (npairs + R));
  sk.part = reg.part;
  sk.flags = reg.flags;
  sk.epoch = reg.epoch;
  sk.slots = static_cast<int>(reg.slots);
  sk.salt = salt;
  return sk;
}

struct FwdWorkspace {
  __nv_bfloat16* act;  // hg (fused) or hn (unfused), [M, d]
  float* part;         // [nt0][M] (fused only)
  SkRegion sk;         // split tails of GEMM0 and GEMM1 (fused only)
};

// CTA-pair tiles of the forward's larger GEMM (sizes the split-tail region)
int64_t fwd_pair_tiles(int64_t M, int64_t d, int64_t N1) {
  return cdiv(M, kPairBM) * std::max(cdiv(d, kBN), cdiv(N1, kBN));
}

// [slot | act | partials | split-tail region]
size_t fwd_ws_bytes(int64_t M, int64_t d, int64_t N1, bool fused) {
  const size_t act = align256(static_cast<size_t>(M) * d * 2);
  const size_t part = fused ? align256(static_cast<size_t>(2 * cdiv(d, kBN)) * M * 4) : 0;
  const size_t sk = fused ? sk_region_bytes(fwd_pair_tiles(M, d, N1)) : 0;
  return kSlotBytes + act + part + sk;
}

enum class FwdKind { kFused, kUnfused, kFusedSwiGLU };

coda_status_t fwd_impl(FwdKind kind, const coda_bf16* x, const coda_bf16* W0, const coda_bf16* z,
                       const coda_bf16* gamma, const coda_bf16* W1, float eps, int64_t M, int64_t d,
                       int64_t N1, coda_bf16* h_out, float* r_out, coda_bf16* y_out,
                       coda_bf16* a_out, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  const bool fused = kind != FwdKind::kUnfused;
  const bool swiglu = kind == FwdKind::kFusedSwiGLU;
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (swiglu && N1 % 16 != 0) return CODA_ERR_UNSUPPORTED_SHAPE;  // N1/2 rows of 16 bytes
  if (M == 0) return CODA_OK;
  if (!x || !W0 || !z || !gamma || !W1 || !h_out || !r_out || (swiglu ? !a_out : !y_out))
    return CODA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {x, W0, z, gamma, W1, h_out, r_out, swiglu ? a_out : y_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (swiglu && !aligned16(y_out)) return CODA_ERR_MISALIGNED;  // optional, may be null
  if (workspace == nullptr || workspace_bytes < fwd_ws_bytes(M, d, N1, fused))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  st = device_setup(&sms, &max_pairs);
  if (st != CODA_OK) return st;
  const bool pair = g_mma_mode.load() == 1;

  FwdWorkspace ws;
  char* const wsb = static_cast<char*>(workspace);
  ws.act = reinterpret_cast<__nv_bfloat16*>(wsb + kSlotBytes);
  ws.part = fused ? reinterpret_cast<float*>(wsb + kSlotBytes +
                                             align256(static_cast<size_t>(M) * d * 2))
                  : nullptr;
  if (fused)
    ws.sk = sk_region(wsb + kSlotBytes + align256(static_cast<size_t>(M) * d * 2) +
                          align256(static_cast<size_t>(2 * cdiv(d, kBN)) * M * 4),
                      fwd_pair_tiles(M, d, N1), wsb);
  const uint64_t salt = next_salt();

  CUtensorMap mA0, mB0, mA1, mB1;
  bool ok = tmap_2d(&mA0, x, d, M, kBK, kBM);           // x  [M, d]  K-major
  ok &= tmap_2d(&mB0, W0, d, d, 64, kBK);               // W0 [d(K), d(N)]  MN-major
  ok &= tmap_2d(&mA1, ws.act, d, M, kBK, kBM);          // hg [M, d]  K-major
  ok &= tmap_2d(&mB1, W1, N1, d, 64, kBK);              // W1 [d(K), N1(N)] MN-major
  if (!ok) return CODA_ERR_LAUNCH;

  const int mt = static_cast<int>(cdiv(M, kBM));
  const int nt0 = static_cast<int>(cdiv(d, kBN));
  const int nt1 = swiglu ? EpiRowScaleSwiGLU::num_col_tiles(static_cast<int>(N1))
                        : static_cast<int>(cdiv(N1, kBN));
  const int Mi = static_cast<int>(M), di = static_cast<int>(d), N1i = static_cast<int>(N1);
  const uint64_t tmo = g_timeout_ns.load();

  EpiResidualGammaSumsq::Params p0 = {};
  p0.z = reinterpret_cast<const __nv_bfloat16*>(z);
  p0.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p0.h_out = reinterpret_cast<__nv_bfloat16*>(h_out);
  p0.hg_out = fused ? ws.act : nullptr;
  p0.part = ws.part;
  const int mtp = static_cast<int>(cdiv(M, kPairBM));
  const int64_t nkb = cdiv(d, kBK);  // k-blocks of both GEMMs (K = d)
  const int np0 = std::min(max_pairs, mtp * nt0), np1 = std::min(max_pairs, mtp * nt1);
  const SkParams sk0 = plan_split_tail(ws.sk, static_cast<int64_t>(mtp) * nt0, np0, nkb, salt);
  const SkParams sk1 = plan_split_tail(ws.sk, static_cast<int64_t>(mtp) * nt1, np1, nkb, salt);
  cudaError_t e =
      pair ? launch(kPairGemm0, 2 * np0, kThreads, kPairGemm0Smem, stream, sk0.epoch != nullptr,
                    mA0, mB0, Mi, di, di, kPairGroupM, p0, sk0, kNoColPlan, tmo)
           : launch(kGemm0, std::min(sms, mt * nt0), kThreads, kGemm0Smem, stream, false, mA0,
                    mB0, Mi, di, di, kGroupM, p0, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  int k_launch = 1;
  FoldedRowReduce fold = {};
  if (fused && g_fold_rowreduce.load() == 1) {
    fold.part = ws.part;
    fold.n_part = 2 * nt0;
    fold.d = di;
    fold.eps = eps;
    fold.r_out = r_out;
  } else if (fused) {
    e = launch(rowreduce_rsqrt_kernel, static_cast<int>(cdiv(M, 256)), 256, 0, stream, false,
               static_cast<const float*>(ws.part), 2 * nt0, Mi, di, eps, r_out);
  } else {
    e = launch(rmsnorm_rows_kernel, Mi, 256, 0, stream, false,
               static_cast<const __nv_bfloat16*>(p0.h_out), p0.gamma, eps, Mi, di, ws.act, r_out);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  if (fold.part == nullptr) after_launch(k_launch++, stream);
  if (swiglu) {
    EpiRowScaleSwiGLU::Params ps = {};
    ps.r = r_out;
    ps.fold = fold;
    ps.y_out = reinterpret_cast<__nv_bfloat16*>(y_out);
    ps.a_out = reinterpret_cast<__nv_bfloat16*>(a_out);
    e = pair ? launch(kPairGemm1Swiglu, 2 * np1, kThreads, kPairGemm1SwigluSmem, stream,
                      sk1.epoch != nullptr, mA1, mB1, Mi, N1i, di, kPairGroupM, ps, sk1, kNoColPlan, tmo)
             : launch(kGemm1Swiglu, std::min(sms, mt * nt1), kThreads, kGemm1SwigluSmem,
                      stream, false, mA1, mB1, Mi, N1i, di, kGroupM, ps, tmo);
  } else {
    EpiRowScale::Params p1 = {};
    p1.r = fused ? r_out : nullptr;
    p1.fold = fold;
    p1.y_out = reinterpret_cast<__nv_bfloat16*>(y_out);
    e = pair ? launch(kPairGemm1, 2 * np1, kThreads, kPairGemm1Smem, stream, sk1.epoch != nullptr,
                      mA1, mB1, Mi, N1i, di, kPairGroupM, p1, sk1, kNoColPlan, tmo)
             : launch(kGemm1, std::min(sms, mt * nt1), kThreads, kGemm1Smem, stream, false, mA1,
                      mB1, Mi, N1i, di, kGroupM, p1, tmo);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(k_launch, stream);
  return CODA_OK;
}

// ---------------------------------------------------------------------------
// Column plans for the CTA-pair data gradient (gemm_pair.cuh, ColPlan).
// ---------------------------------------------------------------------------
// 0: 256-column tiles; 1 (2): the data gradients may use narrower column tiles
// whose widths are multiples of 16 (of 64)
std::atomic<int> g_col_plan{0};
std::atomic<int> g_dgrad_kserp{0};  // 1: the data gradients load every other wave's K backwards

// Most column tiles per row block the data-gradient workspace is sized for.
int64_t dgrad_max_col_tiles(int64_t d) { return 2 * cdiv(d, kBN); }

// Partial slots (each two CTA halves of 128 x 256 fp32) the data-gradient
// workspace holds for the pieces of its last row blocks (PieceWork): three per
// 256 x 256 tile, at most 192 (48 MiB).
int64_t dgrad_piece_slots(int64_t M, int64_t d) {
  return std::min<int64_t>(3 * cdiv(M, kPairBM) * cdiv(d, kBN), 192);
}

// The data gradient's workspace: the 256-byte slot of the launch counter, qpart
// [2 * max tiles][M] fp32, flags [slabs][max tiles] (a launch uses the first
// slabs * nt), then the pieces' partial slots and their flags.
struct DgradWs {
  uint64_t* epoch;
  float* qpart;
  uint64_t* flags;
  float* ppart;      // [pslots][2 CTAs][128 x 256]
  uint64_t* pflags;  // [pslots][2 CTAs]
  int64_t pslots;
};

// [slot | qpart | flags | piece partials | piece flags]
size_t dgrad_ws_bytes(int64_t M, int64_t d) {
  const int64_t slabs = 2 * cdiv(M, kPairBM), nt = dgrad_max_col_tiles(d);
  const int64_t ps = dgrad_piece_slots(M, d);
  return kSlotBytes + align256(static_cast<size_t>(2 * nt) * M * 4) +
         align256(static_cast<size_t>(slabs) * nt * 8) +
         align256(static_cast<size_t>(ps) * 2 * kSkSlotFloats * 4) +
         align256(static_cast<size_t>(ps) * 2 * 8);
}

DgradWs dgrad_ws(void* base, int64_t M, int64_t d) {
  const int64_t slabs = 2 * cdiv(M, kPairBM), nt = dgrad_max_col_tiles(d);
  char* p = static_cast<char*>(base);
  DgradWs w;
  w.epoch = reinterpret_cast<uint64_t*>(p);
  p += kSlotBytes;
  w.qpart = reinterpret_cast<float*>(p);
  p += align256(static_cast<size_t>(2 * nt) * M * 4);
  w.flags = reinterpret_cast<uint64_t*>(p);
  p += align256(static_cast<size_t>(slabs) * nt * 8);
  w.pslots = dgrad_piece_slots(M, d);
  w.ppart = reinterpret_cast<float*>(p);
  p += align256(static_cast<size_t>(w.pslots) * 2 * kSkSlotFloats * 4);
  w.pflags = reinterpret_cast<uint64_t*>(p);
  return w;
}

// ---------------------------------------------------------------------------
// Piece split of the CTA-pair data gradient's last row blocks (gemm_pair.cuh,
// PieceWork).
// ---------------------------------------------------------------------------
std::atomic<int> g_dgrad_pieces{1};  // 1: the planner below may cut the last row blocks

struct PiecePlan {
  int dp_tiles = 0, pieces = 0, lvl_first = 0, lvl = 0;
};

// The k last row blocks (R = k nt tiles, R <= npairs) cut into P pieces of at
// least 16 k-blocks, dealt as PieceWork deals them.  The model counts each
// pair's work in tiles: a whole tile 1, a piece piece_cost / P (for the data
// gradient with the row statistic 1.5: pieces finish later than their share
// of K there, because a pair's last whole tile may wait, holding one of the
// two TMEM accumulators, for its row block's tiles in the next wave, which a
// short piece after it cannot cover; 1.5 fits the GB300 measurements of 14
// shapes, 0.88 to 1.08 of the whole-tile time), plus, for the owners that
// finish the launch, about 2 us per partial they add (a k-block takes about
// 0.33 us).  A plan is taken when it shortens the busiest pair's work by at
// least 3 %.
PiecePlan plan_dgrad_pieces(int mt, int nt, int npairs, int64_t nk, int64_t slots,
                            double piece_cost = 1.5, double min_gain = 0.03) {
  PiecePlan best;
  if (npairs < 2 || nt < 1 || nk < 32) return best;
  const int64_t total = static_cast<int64_t>(mt) * nt;
  const double whole = static_cast<double>((total + npairs - 1) / npairs);
  double best_t = (1.0 - min_gain) * whole;
  for (int k = 1; k <= mt && k * nt <= npairs; ++k) {
    const int64_t R = static_cast<int64_t>(k) * nt, dp = total - R;
    const int64_t W = dp / npairs, E = dp % npairs;
    for (int P = 2; P <= 8 && nk / P >= 16; ++P) {
      if (R * (P - 1) > slots) break;
      int lvl_first = npairs, lvl = 0;
      if (E > 0) {
        lvl_first = static_cast<int>(E);
        lvl = static_cast<int>(std::min<int64_t>(P, (P - 1) * R / (npairs - E)));
      }
      const int64_t rr = R * P - static_cast<int64_t>(npairs - lvl_first) * lvl;
      if (rr < R) continue;
      double mx = 0.0;
      for (int p = 0; p < npairs; ++p) {
        const int64_t pieces = (p >= lvl_first ? lvl : 0) + rr / npairs + (p < rr % npairs ? 1 : 0);
        mx = std::max(mx, static_cast<double>(W + (p < E ? 1 : 0)) + piece_cost * pieces / P);
      }
      const double t = mx + (P - 1) * 6.0 / static_cast<double>(nk);
      if (t < best_t) {
        best_t = t;
        best.dp_tiles = static_cast<int>(dp);
        best.pieces = P;
        best.lvl_first = lvl_first;
        best.lvl = lvl;
      }
    }
  }
  return best;
}

// The piece plan of a CTA-pair data gradient of the given shape on `npairs`
// pairs: the row-statistic launch cuts whole row blocks (a piece counting 1.5
// times its share of K, at least 3 % saved); the tile-local launch of the
// SwiGLU backward cuts any last tiles (a piece counting its share, at least 1 %).
PiecePlan piece_plan_for(int64_t M, int64_t d, int64_t N1, int npairs, bool tile_local) {
  const int mt = static_cast<int>(cdiv(M, kPairBM)), nt = static_cast<int>(cdiv(d, kBN));
  const int64_t nk = cdiv(N1, kBK), slots = dgrad_piece_slots(M, d);
  return tile_local ? plan_dgrad_pieces(mt * nt, 1, npairs, nk, slots, 1.0, 0.01)
                    : plan_dgrad_pieces(mt, nt, npairs, nk, slots);
}

// The piece split's parameters for a row-statistic launch on `npairs` pairs
// (kNoSplitTail when no plan pays or the switch is off).
SkParams dgrad_pieces(const DgradWs& dw, int64_t M, int64_t d, int64_t N1, int npairs,
                      uint64_t salt) {
  SkParams sk = kNoSplitTail;
  if (g_dgrad_pieces.load() == 0) return sk;
  const PiecePlan pp = piece_plan_for(M, d, N1, npairs, false);
  if (pp.pieces == 0) return sk;
  sk.dp_tiles = pp.dp_tiles;
  sk.part = dw.ppart;
  sk.flags = dw.pflags;
  sk.epoch = dw.epoch;
  sk.slots = static_cast<int>(dw.pslots);
  sk.salt = salt;
  sk.pieces = pp.pieces;
  sk.lvl_first = pp.lvl_first;
  sk.lvl = pp.lvl;
  return sk;
}

// Largest per-pair load of a plan with tiles handed out round-robin in
// row-major order, in units of one 256-column tile; `c` is the fixed cost of a
// tile in the same unit.
double plan_load(const ColPlan& cp, int mt, int npairs, double c, std::vector<double>& load) {
  load.assign(npairs, 0.0);
  int64_t t = 0;
  for (int mb = 0; mb < mt; ++mb)
    for (int j = 0; j < cp.nt; ++j, ++t) {
      int n0, width;
      cp.tile(mb, j, n0, width);
      load[t % npairs] += width / 256.0 + c;
    }
  return *std::max_element(load.begin(), load.end());
}

struct PlanKey {
  int64_t mt, d, K;
  int npairs;
  bool operator<(const PlanKey& o) const {
    return std::tie(mt, d, K, npairs) < std::tie(o.mt, o.d, o.K, o.npairs);
  }
};
std::mutex g_plan_mu;
std::map<PlanKey, ColPlan> g_plan_cache;

// The column plan for a data gradient of mt 256-row blocks, d output columns
// and K = N1 on `npairs` CTA pairs: among 256-column tiles and every tiling
// into nt tiles (ceil(d/256) <= nt <= 2 ceil(d/256), at most npairs, so that a
// row block's tiles can all be in flight at once) of widths w and w + step
// (step 16 or 64 as the switch says, w a multiple of step, 128 <= w,
// w + step <= 256), each with its best rotation, the one whose largest
// per-pair load is smallest.  A tile's fixed cost (pipeline fill, drain,
// epilogue not hidden) is taken as 2 us against a pair's 256-column tile time
// 2 * 256 * 256 * K / (25 TFLOP/s); a plan must beat the 256-column tiling by
// 0.5 % to be taken.  Memoised per shape, pair count and step.
ColPlan plan_dgrad_cols(int64_t mt, int64_t d, int64_t K, int npairs) {
  const int mode = g_col_plan.load();
  if (mode == 0 || npairs < 2) return kNoColPlan;
  const int step = mode == 2 ? 64 : 16;
  const PlanKey key{mt, d, K, npairs * 4 + mode};
  {
    std::lock_guard<std::mutex> lock(g_plan_mu);
    auto it = g_plan_cache.find(key);
    if (it != g_plan_cache.end()) return it->second;
  }
  const double c = 2e-6 / (2.0 * 256 * 256 * static_cast<double>(K) / 25e12);
  std::vector<double> load;
  const int nt0 = static_cast<int>(cdiv(d, kBN));
  ColPlan uni = {nt0, kBN, 0, 0, 128, step};
  const double base = plan_load(uni, static_cast<int>(mt), npairs, c, load);
  ColPlan best = kNoColPlan;
  double best_load = base * (1.0 - 0.005);
  const int nt_hi = static_cast<int>(std::min<int64_t>(dgrad_max_col_tiles(d), npairs));
  for (int nt = nt0; nt <= nt_hi; ++nt) {
    int w = static_cast<int>(d / nt) / step * step;
    int nl = static_cast<int>(cdiv(d - static_cast<int64_t>(nt) * w, step));
    if (nl >= nt) {
      w += step;
      nl = 0;
    }
    if (w < 128 || w + (nl > 0 ? step : 0) > kBN) continue;
    for (int rot = 0; rot < (nl > 0 ? nt : 1); ++rot) {
      const ColPlan cp = {nt, w, nl, rot, (w + (nl > 0 ? step : 0)) / 2, step};
      const double l = plan_load(cp, static_cast<int>(mt), npairs, c, load);
      if (l < best_load - 1e-9) {
        best_load = l;
        best = cp;
      }
    }
  }
  std::lock_guard<std::mutex> lock(g_plan_mu);
  g_plan_cache[key] = best;
  return best;
}

// ---------------------------------------------------------------------------
// 8-bit codes with scales (q8.cuh)
// ---------------------------------------------------------------------------
// No tensor of the 8-bit operators has more values than this (several times what a device
// holds), so that byte counts and grids stay far from overflowing.
bool fits(int64_t rows, int64_t cols) { return cols <= (int64_t(1) << 40) / std::max<int64_t>(rows, 1); }

// M rows of n values; n a positive multiple of 8
coda_status_t check_rows(int64_t M, int64_t n) {
  if (M < 0 || n <= 0) return CODA_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if (n % 8 != 0 || M > lim || n > lim || !fits(M, n)) return CODA_ERR_UNSUPPORTED_SHAPE;
  return CODA_OK;
}

// One scale per row: a warp per row up to 1024 columns, a block of up to 1024
// threads holding 4 vectors of 8 values each up to 32768, a block that reads the
// row twice beyond.
template <bool kNorm, bool kRes, bool kH>
cudaError_t launch_row_q8(const RowQ8Params& p, int sms, cudaStream_t stream) {
  const int nvec = p.d / 8;
  if (nvec <= 32)
    return launch(&row_q8_kernel<kNorm, kRes, kH, 1, true>, static_cast<int>(cdiv(p.M, 8)), 256, 0, stream,
                  false, p);
  if (nvec <= 32 * kRowQ8Vec)
    return launch(&row_q8_kernel<kNorm, kRes, kH, kRowQ8Vec, true>, static_cast<int>(cdiv(p.M, 8)), 256,
                  0, stream, false, p);
  const int threads = static_cast<int>(cdiv(nvec, 32 * kRowQ8Vec)) * 32;
  if (threads > 512 && threads <= 1024) {
    // Rows of more than 16384 columns leave one or two blocks to an SM: walked by blocks that stay,
    // where two rows fit and there are at least four for each block (8192 x 28672, norm without a
    // residual 108 us against 139, quantiser 120 against 133; 8192 x 16640, norm with a residual
    // 107 against 160, without 84 against 71; at 8192 x 8192 it is the other way around, 82 us against 74
    // with a residual).
    const int stage = (kRes ? 4 : 2) * p.d;
    const int room = kRingSmem - static_cast<int>(row_ring_bytes(p.d, kNorm, kRes, 0));
    const int stages = std::min(kRingMaxStages, room / stage);
    if (stages >= 2 && p.M >= 4 * static_cast<int64_t>(sms))
      return launch(&row_q8_ring_kernel<kNorm, kRes, kH>, sms, threads,
                    row_ring_bytes(p.d, kNorm, kRes, stages), stream, false, p, stages,
                    g_timeout_ns.load());
  }
  if (threads <= 1024)
    return launch(&row_q8_kernel<kNorm, kRes, kH, kRowQ8Vec, false>, p.M, threads, 0, stream, false, p);
  return launch(&row_q8_kernel<kNorm, kRes, kH, 0, false>, p.M, 1024, 0, stream, false, p);
}

// Grid of the kernels on blocks of 128 columns: x over rows, y over a row's blocks.
// `lanes` of them share a block of 128 columns.
bool q8_block_grid(int64_t M, int64_t n, int lanes, dim3* grid) {
  const int64_t nb = cdiv(n, kQ8Block);
  const int lg = q8_span_log2(static_cast<int>(std::min<int64_t>(nb, 16)));
  const int64_t gx = cdiv(M, kQ8Passes * ((256 / lanes) >> lg)), gy = cdiv(nb, int64_t(1) << lg);
  if (gx > 0x7fffffff || gy > 65535) return false;
  *grid = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  return true;
}

coda_status_t check_product(int64_t M, int64_t K, int64_t N) {
  if (M < 0 || K <= 0 || N <= 0) return CODA_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  // 16-byte rows of one-byte codes
  if (K % 16 != 0 || N % 16 != 0 || M > lim || K > lim || N > lim || !fits(M, K) || !fits(K, N) ||
      !fits(M, N))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  return CODA_OK;
}

// Blocks along K (a cluster) of the few-token product: as many as one wave of `slots`
// blocks holds.  A wave more costs more than the idle slots (N = 28672, K = 4096, one token:
// 224 blocks 25 us, 448 in two waves 28 us, 896 33 us; N = 4096: 32 blocks 12 us, 256 7 us).
// `most`: blocks of the largest cluster that fits.
int small_split(int64_t K, int64_t N, int slots, int most) {
  const int64_t tiles = cdiv(N, kSmallChannels), steps = cdiv(K, kSmallStep);
  int s = 1;
  while (s < most && tiles * s * 2 <= slots && steps >= 2 * s * kSmallWarps) s *= 2;
  return s;
}

int small_groups(int64_t M) { return M <= 8 ? 1 : M <= 16 ? 2 : 4; }

cudaError_t launch_product_small(const SmallQ8Params& p, const uint8_t* a_q, const uint8_t* W_q,
                                 int split, cudaStream_t stream) {
  const int groups = small_groups(p.M);
  CUtensorMap mW, mA;
  if (!tmap_2d_u8(&mW, W_q, p.N, p.K, kSmallChannels, kSmallStep) ||
      !tmap_2d_u8(&mA, a_q, p.K, p.M, kSmallStep, 8 * groups, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int64_t grid = cdiv(p.N, kSmallChannels) * split;
  auto* const kernel = groups == 1 ? kProductSmall1 : groups == 2 ? kProductSmall2 : kProductSmall4;
  const uint32_t smem = groups == 1   ? SmallSmem<1>::kBytes
                        : groups == 2 ? SmallSmem<2>::kBytes
                                      : SmallSmem<4>::kBytes;
  return launch_cluster(kernel, static_cast<int>(grid), 32 * kSmallWarps, smem, stream, false, split,
                        mW, mA, p, split, g_timeout_ns.load());
}

// The INT8 product's three kernels.
//   few tokens (q8_small.cuh)    up to 8 tokens; more while W is small, where it starts sooner.  Against
//                                the mid-size kernel, 16 tokens: W of 17 MB 9.0 us and 10.4, 59 MB 16.5
//                                and 16.9, 117 MB 29.2 and 27.1; 32 tokens: 17 MB 9.8 and 11.4, 59 MB
//                                19.3 and 17.5
//   mid-size (q8_mid.cuh)        up to kMidSure tokens, and beyond while its estimate is the lower one
//   whole GEMM                   a and W widened to bf16 in the workspace first
constexpr int64_t kMidSure = 1024;  // 1025 x 4096 x 14336: 89 us against 114

bool product_small(int64_t M, int64_t K, int64_t N) {
  return M <= 8 || (M <= 16 && K * N < (int64_t(5) << 24)) ||
         (M <= kSmallMaxTokens && K * N < (int64_t(3) << 24));
}

// Time of the whole-GEMM form: widening at 6.2 bytes per ps (1 read, 2 written per code), waves
// of 256 x 256 tiles at 333 ns per 64 rows of K, about 7 us of launches and ends.
double product_gemm_ns(int64_t M, int64_t K, int64_t N, int pairs) {
  return 3.0 * (static_cast<double>(M) * K + static_cast<double>(K) * N) / 6200.0 +
         333.0 * static_cast<double>(cdiv(cdiv(M, kPairBM) * cdiv(N, kBN), pairs) * cdiv(K, kBK)) +
         7000.0;
}

// Tokens per CTA pair, pairs along K and blocks per SM of the mid-size product: those with the
// least estimated time, waves of clusters times a cluster's (no tokens where not even a pair fits); more token tiles only where they gain
// 5 %, as each reads W again.  Fitted to sweeps on GB300 (its picks are 1 % above the best on the
// average of 40 shapes): a step of 64 rows takes 1.33 ns per token (the tensor cores), below about
// 300 tokens 235 ns and 0.53 ns per token (the way from a stage to a slot) and no less than with 64,
// two blocks on an SM 364 ns and 1.09 ns per token for both; a pair's start and its sums'
// way out 3 us and 5 ns per token, a split's exchange 0.5 us and 10 ns more, of four pairs or
// with two blocks on an SM 1 us and 25 ns.
struct MidPlan {
  int tokens, split;
  bool narrow;
  double ns;
};

MidPlan plan_mid(int64_t M, int64_t K, int64_t N, const int (*clusters)[3]) {
  const int64_t ct = cdiv(N, 2 * kMidChannels), nk = cdiv(K, kMidK);
  MidPlan best = {0, 1, false, 1e30};
  const int64_t mt0 = cdiv(M, kMidMaxTokens);
  for (int64_t mt = mt0; mt <= mt0 + 3; ++mt) {
    int64_t tokens = cdiv(cdiv(M, mt), 16) * 16;
    if (tokens > 256) tokens = cdiv(tokens, 32) * 32;
    const double t = static_cast<double>(tokens);
    for (int i = 0, s = 1; s <= kMidMaxSplit; ++i, s *= 2) {
      if ((s > 1 && nk < 4 * s) || clusters[0][i] == 0) break;
      const int64_t tiles = ct * cdiv(M, tokens);
      for (int narrow = 0; narrow < 2; ++narrow) {
        // a narrow block alone on its SM is a wide one with shorter rings
        if (narrow && (tokens > MidShape<true>::kTokens || tiles <= clusters[0][i])) break;
        const double t64 = std::max(t, 64.0);
        const double step = narrow ? 364.0 + 1.09 * t64 : std::max(1.33 * t, 235.0 + 0.53 * t64);
        const double exchange =
            s == 1 ? 0.0 : s == 4 || narrow ? 1000.0 + 25.0 * t : 500.0 + 10.0 * t;
        const double pair = static_cast<double>(cdiv(nk, s)) * step + 3000.0 + 5.0 * t + exchange;
        const double ns = static_cast<double>(cdiv(tiles, clusters[narrow][i])) * pair;
        if (ns < 0.95 * best.ns) best = {static_cast<int>(tokens), s, narrow != 0, ns};
      }
    }
  }
  return best;
}

enum ProductForm { kFormNone, kFormSmall, kFormMid, kFormGemm };

struct ProductPlan {
  ProductForm form;
  int split;    // blocks (few tokens) or pairs (mid-size) along K
  MidPlan mid;  // mid-size
};

// The form of a product on a device of `sms` SMs, `pairs` co-resident CTA pairs of the GEMM and so
// many clusters of the mid-size form; none where that form is needed and does not fit.
ProductPlan plan_product(int64_t M, int64_t K, int64_t N, int sms, int pairs,
                         const int (*clusters)[3]) {
  ProductPlan p = {kFormNone, 1, {}};
  if (product_small(M, K, N)) {
    const int most = clusters[0][2] > 0 ? 8 : clusters[0][1] > 0 ? 4 : clusters[0][0] > 0 ? 2 : 1;
    p.form = kFormSmall;
    p.split = small_split(K, N, small_groups(M) <= 2 ? 2 * sms : sms, most);
    return p;
  }
  p.mid = plan_mid(M, K, N, clusters);
  p.split = p.mid.split;
  // (short K, whose waves the plan takes for some 3 us shorter than they are: 10 % in hand)
  if (p.mid.tokens > 0 &&
      (M <= kMidSure || 1.1 * p.mid.ns < product_gemm_ns(M, K, N, std::max(pairs, 1))))
    p.form = kFormMid;
  else if (M > kMidSure)
    p.form = kFormGemm;
  return p;
}

cudaError_t launch_product_mid(MidQ8Params p, const uint8_t* a_q, const uint8_t* W_q,
                               const MidPlan& plan, cudaStream_t stream) {
  p.tokens = plan.tokens;
  p.split = plan.split;
  p.parts = p.tokens > 256 ? 2 : 1;
  p.tok_warps = std::min(plan.narrow ? 2 : 4, static_cast<int>(cdiv(p.tokens, 64)));
  // As many slots as tensor memory holds and as leave six stages; the stages have the rest.
  const int rings = static_cast<int>(plan.narrow ? MidShape<true>::kRings : MidShape<false>::kRings);
  const int cols = static_cast<int>(plan.narrow ? MidShape<true>::kCols : MidShape<false>::kCols);
  const int stage = static_cast<int>(mid_stage_bytes(p.tokens));
  const int slot = static_cast<int>(mid_slot_bytes(p.tokens));
  p.pairs_slots = std::min({kMidMaxSlots, (cols - (p.tokens + 31) / 32 * 32) / 32,
                            (rings - 6 * stage) / slot}) / 2;
  p.pairs_stages = std::min(kMidMaxStages, (rings - 2 * p.pairs_slots * slot) / stage) / 2;
  CUtensorMap mW, mX;
  if (!tmap_2d_u8(&mW, W_q, p.N, p.K, kMidChannels, kMidK) ||
      !tmap_2d_u8(&mX, a_q, p.K, p.M, kMidK, p.tokens / p.parts / 2, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const int64_t grid = cdiv(p.N, 2 * kMidChannels) * cdiv(p.M, p.tokens) * 2 * p.split;
  const cudaError_t e = launch_cluster(
      plan.narrow ? kProductNarrow : kProductMid, static_cast<int>(grid), mid_threads(plan.narrow),
      plan.narrow ? MidShape<true>::kBytes : MidShape<false>::kBytes, stream, false, 2 * p.split, mW, mX,
      p, g_timeout_ns.load());
  if (e == cudaSuccess) after_launch(0, stream);
  return e;
}

// ---------------------------------------------------------------------------
// The 8-bit paged cache (cache_q8.cuh, attn_q8.cuh)
// ---------------------------------------------------------------------------
constexpr int kFewRows = 16;  // of its largest tile
// Packed rows of a sequence that go to the kernel for few.  Measured, few / tiles: 64 sequences over 8000 keys, 8 key heads of
// 128, 32 rows 353 / 454 us, 40 515 / 455, 64 682 / 457; 16 over 3000, 4 of 64, 40 rows 34 / 43, 64 41 / 43, 128 66 / 43; 4
// over 1000, 8 of 128, 40 rows 24 / 30, 64 25 / 30, 128 34 / 31.  The border is at 32 rows where the keys' bytes are the
// bound and near 100 where latency is: one in between.
constexpr int kFewMost = 48;
constexpr int64_t kMaxSequences = 8192, kMaxHeads = 1024;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

coda_status_t check_heads(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D) {
  if (T < 0 || B < 0 || Hq <= 0 || Hk <= 0 || D <= 0) return CODA_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  if ((D != 64 && D != 128) || Hq % Hk != 0 || Hq > kMaxHeads || B > kMaxSequences || T > lim / Hq ||
      !fits(T, (Hq + 2 * Hk) * D))
    return CODA_ERR_UNSUPPORTED_SHAPE;
  return CODA_OK;
}

// The sizes, then the pointers of the cache and of the batch (not looked at where nothing is to do).
coda_status_t check_cache(const int8_t* k_q, const float* k_s, const int8_t* v_q, const float* v_s,
                          int64_t pages, int64_t Hq, int64_t Hk, int64_t page, int64_t D,
                          const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t B,
                          int64_t width, int64_t T, CacheQ8* c, BatchQ8* bt) {
  const coda_status_t st = check_heads(T, B, Hq, Hk, D);
  if (st != CODA_OK) return st;
  if (pages <= 0 || page <= 0 || width <= 0) return CODA_ERR_INVALID_ARG;
  const int64_t lim = (int64_t(1) << 31) - 256;
  // (a token's number, and the pages of all sequences, stay far below 2^31)
  if (page < 16 || page > 256 || (page & (page - 1)) != 0 || pages > lim || !fits(pages, Hk * page * D) ||
      width > (int64_t(1) << 30) / page)
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || B == 0) return CODA_OK;
  const void* ptrs[] = {k_q, k_s, v_q, v_s};
  for (const void* p : ptrs)
    if (!p) return CODA_ERR_INVALID_ARG;
  if (!cu || !lens || !table) return CODA_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (!aligned4(cu) || !aligned4(lens) || !aligned4(table)) return CODA_ERR_MISALIGNED;
  c->k_q = reinterpret_cast<uint8_t*>(const_cast<int8_t*>(k_q));
  c->k_s = const_cast<float*>(k_s);
  c->v_q = reinterpret_cast<uint8_t*>(const_cast<int8_t*>(v_q));
  c->v_s = const_cast<float*>(v_s);
  c->pages = static_cast<int>(pages);
  c->Hk = static_cast<int>(Hk);
  c->page_log2 = 0;
  while ((int64_t(1) << c->page_log2) < page) ++c->page_log2;
  bt->cu = cu;
  bt->lens = lens;
  bt->table = table;
  bt->B = static_cast<int>(B);
  bt->width = static_cast<int>(width);
  bt->rows = static_cast<int>(T);
  return CODA_OK;
}

// The part of x that is no whole number, in -1/2 .. 1/2 (exact), in steps of 2^-64, modulo 2^64
uint64_t fraction64(double x) {
  const double part = (x - std::nearbyint(x)) * 0x1p64;  // -2^63 .. 2^63
  return part < 0x1p63 ? static_cast<uint64_t>(std::llrint(part)) : uint64_t(1) << 63;
}

// turn[i]: inv_freq[i] / (2 pi) modulo one turn, a turn being 2^64.  1 / (2 pi) is the sum of two doubles, 2^-110 off, and
// its product with a frequency of two more, so that a turn is off by a step or less: a double's own 2^-54 of a turn would be
// 2^-23 of one at positions near 2^31.
coda_status_t rope_of(const double* inv_freq, const int32_t* axis, int64_t half, const int32_t* pos,
                      int64_t axes, int pairs, int64_t D, RopeQ8* r) {
  if (half < 0 || axes < 1 || axes > kRopeAxes || (pos == nullptr && axes != 1)) return CODA_ERR_INVALID_ARG;
  if (half % 8 != 0 || 2 * half > D) return CODA_ERR_UNSUPPORTED_SHAPE;
  if (half > 0 && inv_freq == nullptr) return CODA_ERR_INVALID_ARG;
  if (!aligned4(pos)) return CODA_ERR_MISALIGNED;
  *r = RopeQ8{};
  for (int64_t i = 0; i < half; ++i) {
    if (!std::isfinite(inv_freq[i])) return CODA_ERR_INVALID_ARG;
    if (axis != nullptr && (axis[i] < 0 || axis[i] >= axes)) return CODA_ERR_INVALID_ARG;
    constexpr double kHigh = 0.15915494309189535, kLow = -9.839338337591243e-18;
    const double f = inv_freq[i], turns = f * kHigh, rest = std::fma(f, kHigh, -turns) + f * kLow;
    r->turn[i] = fraction64(turns) + fraction64(rest);
    r->axis[i] = static_cast<uint8_t>(axis != nullptr ? axis[i] : 0);
  }
  r->pos = pos;
  r->half = static_cast<int>(half);
  r->pairs = pairs != 0;
  return CODA_OK;
}

// Parts of the attention's items: [cuts | maxima and sums | units | outputs], two parts per block, of as many rows as
// a tile may have (`rows`: packed rows of the call at most)
int attn_ws_rows(int tile_rows, int64_t rows) { return static_cast<int>(std::min<int64_t>(tile_rows, rows)); }

size_t attn_ws_bytes(int tile_rows, int64_t rows, int64_t D) {
  const size_t parts = size_t(2) * kAttnMaxBlocks * attn_ws_rows(tile_rows, rows);
  return align256(kAttnMaxBlocks * sizeof(AttnCutFew)) + align256(parts * sizeof(float2)) + align256(parts * sizeof(float)) +
         align256(parts * D * sizeof(float));
}

AttnWs attn_ws(char* at, int tile_rows, int64_t rows, int64_t D) {
  AttnWs w;
  w.tile = tile_rows;
  w.rows = attn_ws_rows(tile_rows, rows);
  w.cut = reinterpret_cast<AttnCutFew*>(at);
  at += align256(kAttnMaxBlocks * sizeof(AttnCutFew));
  w.ml = reinterpret_cast<float2*>(at);
  at += align256(size_t(2) * kAttnMaxBlocks * w.rows * sizeof(float2));
  w.unit = reinterpret_cast<float*>(at);
  at += align256(size_t(2) * kAttnMaxBlocks * w.rows * sizeof(float));
  w.o = reinterpret_cast<float*>(at);
  return w;
}

// Sequences of up to kFewMost packed rows go to the kernel for few, the others to the one for tiles, each with
// its own share of the blocks; one join serves both.  Without a hint of `rows` (the most of a sequence) both
// run, and one of them may find nothing (64 single tokens over 8000 keys: 164 us, 159 with the hint); a single sequence goes to
// tiles if it may have more than a few rows.  If a sequence has more rows than the hint says, the kernel for few takes it.
//
// Its tiles are of 8 rows where no sequence has more; else of 16, which read a key once where tiles of 8 read it twice (64
// sequences of six tokens of 8 heads over 3000 keys: 240 us with the hint).  Beside tiles the short sequences' rows are not
// known: with a hint they are taken for single tokens (two chunks beside four: 139 us, 143 with tiles of 16; beside 16
// drafts of five 176 and 171), without one where there are as many rows as sequences (64 single tokens: 164 us, 193 with
// tiles of 16), and not where there are more (the drafts of six: 247 us, 356 with tiles of 8).
template <int kD>
cudaError_t launch_attn(const AttnQ8Params& p, char* at, int64_t rows, bool hint, int blocks, cudaStream_t stream) {
  const bool tiles = rows > kFewMost, few = !tiles || p.batch.B > 1;
  const int64_t all = static_cast<int64_t>(p.batch.rows) * p.group;  // (a hint may be too small)
  const bool eight = rows <= 8 || (tiles && p.group <= 8 && (hint || p.batch.rows <= p.batch.B));
  const AttnWs wf = attn_ws(at, eight ? 8 : kFewRows, all, kD);
  const AttnWs wt = attn_ws(at + attn_ws_bytes(kFewRows, all, kD), kTileRows, kTileRows, kD);
  int k = 0;
  cudaError_t e = cudaSuccess;
  if (few) {
    const AttnDeal deal = {0, tiles ? kFewMost : 0x7fffffff};
    e = eight ? launch(&attn_q8_few_kernel<kD, 1>, blocks, FewDeal<1>::kThreads, FewSmem<kD, 1>::kBytes, stream, false, p, wf,
                       deal)
              : launch(&attn_q8_few_kernel<kD, 2>, blocks, FewDeal<2>::kThreads, FewSmem<kD, 2>::kBytes, stream, false, p, wf,
                       deal);
    if (e == cudaSuccess) after_launch(k++, stream);
  }
  if (e == cudaSuccess && tiles) {
    e = launch(&attn_q8_tile_kernel<kD>, blocks, kTileThreads, TileSmem<kD>::kBytes, stream, false, p, wt,
               AttnDeal{few ? kFewMost : 0, 0x7fffffff}, g_timeout_ns.load());
    if (e == cudaSuccess) after_launch(k++, stream);
  }
  if (e == cudaSuccess) {
    e = launch(&attn_q8_join_kernel<kD>, dim3(blocks, (few ? 1 : 0) + (tiles ? kTileRows / 16 : 0)), 256, 0, stream, false,
               p, wf, wt, few ? 0 : 1, blocks);
    if (e == cudaSuccess) after_launch(k++, stream);
  }
  return e;
}

template <int kD>
cudaError_t launch_cache_write(const CacheWriteParams& p, const RopeQ8& r, int sms, cudaStream_t stream) {
  const int T = p.batch.rows, heads = p.Hq + 2 * p.cache.Hk;
  // four tokens to a block while that leaves every SM some; else one, its heads over several blocks
  if (T >= 8 * sms)
    return launch(&cache_write_q8_kernel<kD, 4>, static_cast<int>(cdiv(T, 4)), kCacheThreads, 0, stream,
                  false, p, r);
  const int64_t most = cdiv(heads, kCacheThreads / (kD / 8));
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(most, 4 * sms / T));
  return launch(&cache_write_q8_kernel<kD, 1>, dim3(T, static_cast<unsigned>(parts)), kCacheThreads, 0,
                stream, false, p, r);
}

template <int kD>
cudaError_t launch_cache_read(const CacheReadParams& p, int sms, cudaStream_t stream) {
  const int64_t blocks = cdiv(p.batch.rows, kReadTokens);
  const int64_t most = cdiv(kReadTokens * p.cache.Hk, kCacheThreads / (kD / 16));
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(most, 4 * sms / blocks));
  return launch(&cache_read_q8_kernel<kD>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(parts)),
                kCacheThreads, 0, stream, false, p);
}

}  // namespace

extern "C" {

size_t coda_fwd_workspace_bytes(int64_t M, int64_t d, int64_t N1) {
  if (check_common(M, d, N1) != CODA_OK || M == 0) return 0;
  return fwd_ws_bytes(M, d, N1, true);
}

size_t coda_fwd_unfused_workspace_bytes(int64_t M, int64_t d, int64_t N1) {
  if (check_common(M, d, N1) != CODA_OK || M == 0) return 0;
  return fwd_ws_bytes(M, d, N1, false);
}

size_t coda_bwd_dgrad_workspace_bytes(int64_t M, int64_t d, int64_t N1) {
  if (check_common(M, d, N1) != CODA_OK || M == 0) return 0;
  // one flag per (128-row slab, column tile); CTA-pair tiles cover 2 * ceil(M/256) slabs
  // and a column plan cuts a row block into at most twice ceil(d/256) tiles; then the
  // launch counter's 256-byte slot
  return dgrad_ws_bytes(M, d);
}

coda_status_t coda_fwd(const coda_bf16* x, const coda_bf16* W0, const coda_bf16* z,
                       const coda_bf16* gamma, const coda_bf16* W1, float eps, int64_t M, int64_t d,
                       int64_t N1, coda_bf16* h_out, float* r_out, coda_bf16* y_out,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return fwd_impl(FwdKind::kFused, x, W0, z, gamma, W1, eps, M, d, N1, h_out, r_out, y_out,
                  nullptr, workspace, workspace_bytes, stream);
}

coda_status_t coda_fwd_swiglu(const coda_bf16* x, const coda_bf16* W0, const coda_bf16* z,
                              const coda_bf16* gamma, const coda_bf16* W1, float eps, int64_t M,
                              int64_t d, int64_t N1, coda_bf16* h_out, float* r_out,
                              coda_bf16* y_out, coda_bf16* a_out, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  return fwd_impl(FwdKind::kFusedSwiGLU, x, W0, z, gamma, W1, eps, M, d, N1, h_out, r_out, y_out,
                  a_out, workspace, workspace_bytes, stream);
}

coda_status_t coda_fwd_unfused(const coda_bf16* x, const coda_bf16* W0, const coda_bf16* z,
                               const coda_bf16* gamma, const coda_bf16* W1, float eps, int64_t M,
                               int64_t d, int64_t N1, coda_bf16* h_out, float* r_out,
                               coda_bf16* y_out, void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  return fwd_impl(FwdKind::kUnfused, x, W0, z, gamma, W1, eps, M, d, N1, h_out, r_out, y_out,
                  nullptr, workspace, workspace_bytes, stream);
}

coda_status_t coda_bwd_dgrad(const coda_bf16* dy, const coda_bf16* W1, const coda_bf16* h,
                             const float* r, const coda_bf16* gamma, int64_t M, int64_t d,
                             int64_t N1, coda_bf16* dh_out, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (M == 0) return CODA_OK;
  if (!dy || !W1 || !h || !r || !gamma || !dh_out) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, W1, h, r, gamma, dh_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (workspace == nullptr || workspace_bytes < coda_bwd_dgrad_workspace_bytes(M, d, N1))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  st = device_setup(&sms, &max_pairs);
  if (st != CODA_OK) return st;
  const bool pair = g_mma_mode.load() == 1;

  // Row-major tile order; every column tile of a row block must be in flight
  // at once (at most one wave per row block), see EpiRmsNormBackward.
  const int mt = static_cast<int>(cdiv(M, pair ? kPairBM : kBM));
  ColPlan cp = pair ? plan_dgrad_cols(mt, d, N1, max_pairs) : kNoColPlan;
  cp.kserp = g_dgrad_kserp.load();
  const int nt = cp.nt > 0 ? cp.nt : static_cast<int>(cdiv(d, kBN));
  int units = pair ? std::min(max_pairs, mt * nt) : std::min(sms, mt * nt);
  if (nt > units) return CODA_ERR_UNSUPPORTED_SHAPE;

  CUtensorMap mA, mB;
  bool ok = tmap_2d(&mA, dy, N1, M, kBK, kBM);                  // dy [M, N1] K-major (K = N1)
  ok &= tmap_2d(&mB, W1, N1, d, kBK, pair ? cp.b_rows : kBN);   // W1 [d(N), N1(K)] K-major
  if (!ok) return CODA_ERR_LAUNCH;

  const DgradWs dw = dgrad_ws(workspace, M, d);
  const uint64_t salt = next_salt();
  // the last row blocks cut into K pieces, when the planner finds it pays (every pair runs)
  const SkParams sk =
      (pair && cp.nt == 0) ? dgrad_pieces(dw, M, d, N1, max_pairs, salt) : kNoSplitTail;
  if (sk.pieces > 0) units = max_pairs;
  EpiRmsNormBackward::Params p = {};
  p.h = reinterpret_cast<const __nv_bfloat16*>(h);
  p.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p.r = r;
  p.dh_out = reinterpret_cast<__nv_bfloat16*>(dh_out);
  p.qpart = dw.qpart;
  p.flags = dw.flags;
  p.epoch = dw.epoch;
  p.salt = salt;
  cudaError_t e =
      pair ? launch(kPairDgrad, 2 * units, kThreads, kPairDgradSmem, stream, true, mA, mB,
                    static_cast<int>(M), static_cast<int>(d), static_cast<int>(N1), 1, p, sk, cp,
                    g_timeout_ns.load())
           : launch(kDgrad, units, kThreads, kDgradSmem, stream, true, mA, mB,
                    static_cast<int>(M), static_cast<int>(d), static_cast<int>(N1), 1, p,
                    g_timeout_ns.load());
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

size_t coda_fwd_fp8_workspace_bytes(int64_t M, int64_t d, int64_t N1) {
  if (check_common(M, d, N1) != CODA_OK || M == 0) return 0;
  return kSlotBytes + align256(static_cast<size_t>(M) * d) +
         align256(static_cast<size_t>(2 * cdiv(d, kBN)) * M * 4);
}

coda_status_t coda_fwd_fp8(const uint8_t* x_q, float sx, const uint8_t* W0_q, float sW0,
                           const coda_bf16* z, const coda_bf16* gamma, const uint8_t* W1_q,
                           float sW1, float s_hg, float eps, int64_t M, int64_t d, int64_t N1,
                           coda_bf16* h_out, float* r_out, coda_bf16* y_out, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (d % 16 != 0 || N1 % 16 != 0) return CODA_ERR_UNSUPPORTED_SHAPE;  // 16-byte FP8 rows
  if (M == 0) return CODA_OK;
  if (!x_q || !W0_q || !z || !gamma || !W1_q || !h_out || !r_out || !y_out)
    return CODA_ERR_INVALID_ARG;
  const float scales[] = {sx, sW0, sW1, s_hg};
  for (float v : scales)
    if (!std::isfinite(v) || !(v > 0.f)) return CODA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {x_q, W0_q, z, gamma, W1_q, h_out, r_out, y_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (workspace == nullptr || workspace_bytes < coda_fwd_fp8_workspace_bytes(M, d, N1))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  st = device_setup(&sms, &max_pairs);
  if (st != CODA_OK) return st;
  const uint64_t tmo = g_timeout_ns.load();
  const int Mi = static_cast<int>(M), di = static_cast<int>(d), N1i = static_cast<int>(N1);
  uint8_t* hq = static_cast<uint8_t*>(workspace) + kSlotBytes;
  float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSlotBytes +
                                         align256(static_cast<size_t>(M) * d));

  CUtensorMap mA0, mB0, mA1, mB1;
  bool ok = tmap_2d_u8(&mA0, x_q, d, M, 128, 128);    // x  [M, d] codes, K-major
  ok &= tmap_2d_u8(&mB0, W0_q, d, d, 128, 128);       // W0 [d(K), d(N)], MN-major
  ok &= tmap_2d_u8(&mA1, hq, d, M, 128, 128);         // hq [M, d], K-major
  ok &= tmap_2d_u8(&mB1, W1_q, N1, d, 128, 128);      // W1 [d(K), N1(N)], MN-major
  if (!ok) return CODA_ERR_LAUNCH;

  const int mtp = static_cast<int>(cdiv(M, kPairBM));
  const int nt0 = static_cast<int>(cdiv(d, kBN));
  const int nt1 = static_cast<int>(cdiv(N1, kBN));
  EpiResidualGammaSumsqFp8::Params p0 = {};
  p0.z = reinterpret_cast<const __nv_bfloat16*>(z);
  p0.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p0.h_out = reinterpret_cast<__nv_bfloat16*>(h_out);
  p0.hq_out = hq;
  p0.part = part;
  p0.acc_scale = sx * sW0;
  p0.inv_s_hg = 1.0f / s_hg;
  cudaError_t e = launch(kPairGemm0F8, 2 * std::min(max_pairs, mtp * nt0), kThreads,
                         kPairGemm0F8Smem, stream, false, mA0, mB0, Mi, di, di, kPairGroupM, p0, kNoSplitTail,
                         kNoColPlan, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  e = launch(rowreduce_rsqrt_kernel, static_cast<int>(cdiv(M, 256)), 256, 0, stream, false,
             static_cast<const float*>(part), 2 * nt0, Mi, di, eps, r_out);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(1, stream);
  EpiRowScaleFp8::Params p1 = {};
  p1.r = r_out;
  p1.y_out = reinterpret_cast<__nv_bfloat16*>(y_out);
  p1.scale = s_hg * sW1;
  e = launch(kPairGemm1F8, 2 * std::min(max_pairs, mtp * nt1), kThreads, kPairGemm1F8Smem, stream,
             false, mA1, mB1, Mi, N1i, di, kPairGroupM, p1, kNoSplitTail, kNoColPlan, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(2, stream);
  return CODA_OK;
}

// CTA-pair tiles of the full backward's largest split-capable GEMM (dW1, dx or
// dW0), which sizes its split-tail region
int64_t bwd_pair_tiles(int64_t M, int64_t d, int64_t N1) {
  return std::max(cdiv(d, kPairBM) * cdiv(std::max(d, N1), kBN), cdiv(M, kPairBM) * cdiv(d, kBN));
}

size_t coda_bwd_workspace_bytes(int64_t M, int64_t d, int64_t N1) {
  if (check_common(M, d, N1) != CODA_OK || M == 0) return 0;
  const int64_t slabs = std::max(2 * cdiv(M, kPairBM), cdiv(M, kBM));
  return coda_bwd_dgrad_workspace_bytes(M, d, N1) + align256(static_cast<size_t>(M) * d * 2) +
         align256(static_cast<size_t>(4 * slabs) * d * 4) + sk_region_bytes(bwd_pair_tiles(M, d, N1));
}

coda_status_t coda_bwd(const coda_bf16* dy, const coda_bf16* x, const coda_bf16* W0,
                       const coda_bf16* W1, const coda_bf16* h, const float* r,
                       const coda_bf16* gamma, const coda_bf16* dh_res, int64_t M, int64_t d,
                       int64_t N1, coda_bf16* dh_out, coda_bf16* dx_out, float* dgamma_out,
                       float* dW0_out, float* dW1_out, void* workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (M == 0) return CODA_OK;
  if (!dy || !x || !W0 || !W1 || !h || !r || !gamma || !dh_out || !dx_out || !dgamma_out ||
      !dW0_out || !dW1_out)
    return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, x, W0, W1, h, r, gamma, dh_out, dx_out, dgamma_out, dW0_out, dW1_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (dh_res != nullptr && !aligned16(dh_res)) return CODA_ERR_MISALIGNED;
  if (workspace == nullptr || workspace_bytes < coda_bwd_workspace_bytes(M, d, N1))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  st = device_setup(&sms, &max_pairs);
  if (st != CODA_OK) return st;
  const bool pair = g_mma_mode.load() == 1;
  const uint64_t tmo = g_timeout_ns.load();
  const int Mi = static_cast<int>(M), di = static_cast<int>(d), N1i = static_cast<int>(N1);

  const int nt = static_cast<int>(cdiv(d, kBN));  // 256-column tiles of the GEMMs with N = d
  const int mt = static_cast<int>(cdiv(M, pair ? kPairBM : kBM));
  // launch 1 (the data gradient) may cut its row blocks into a column plan's tiles
  ColPlan cp = pair ? plan_dgrad_cols(mt, d, N1, max_pairs) : kNoColPlan;
  cp.kserp = g_dgrad_kserp.load();
  const int nt1 = cp.nt > 0 ? cp.nt : nt;
  int units = pair ? std::min(max_pairs, mt * nt1) : std::min(sms, mt * nt1);
  if (nt1 > units) return CODA_ERR_UNSUPPORTED_SHAPE;
  const int slabs = pair ? 2 * mt : mt;

  char* ws = static_cast<char*>(workspace);
  const DgradWs dw = dgrad_ws(ws, M, d);
  char* rest = ws + coda_bwd_dgrad_workspace_bytes(M, d, N1);
  __nv_bfloat16* h2 = reinterpret_cast<__nv_bfloat16*>(rest);
  float* gpart = reinterpret_cast<float*>(rest + align256(static_cast<size_t>(M) * d * 2));
  const SkRegion skr =
      sk_region(rest + align256(static_cast<size_t>(M) * d * 2) +
                    align256(static_cast<size_t>(4 * std::max(2 * cdiv(M, kPairBM), cdiv(M, kBM))) *
                             d * 4),
                bwd_pair_tiles(M, d, N1), dw.epoch);
  const uint64_t salt = next_salt();

  const uint32_t bbox = pair ? 128 : kBN;
  CUtensorMap mDy, mW1, mH2, mDyMN, mDh, mW0, mX, mDhMN;
  bool ok = tmap_2d(&mDy, dy, N1, M, kBK, kBM);     // dy [M, N1] K-major (dgrad)
  ok &= tmap_2d(&mW1, W1, N1, d, kBK, pair ? cp.b_rows : kBN);  // W1 [d(N), N1(K)] K-major
  ok &= tmap_2d(&mH2, h2, d, M, 64, kBK);           // h2^T: [M(K), d(M)] MN-major A
  ok &= tmap_2d(&mDyMN, dy, N1, M, 64, kBK);        // dy: [M(K), N1(N)] MN-major B
  ok &= tmap_2d(&mDh, dh_out, d, M, kBK, kBM);      // dh [M, d] K-major A
  ok &= tmap_2d(&mW0, W0, d, d, kBK, bbox);         // W0 [d_in(N), d_out(K)] K-major B
  ok &= tmap_2d(&mX, x, d, M, 64, kBK);             // x^T: [M(K), d(M)] MN-major A
  ok &= tmap_2d(&mDhMN, dh_out, d, M, 64, kBK);     // dh: [M(K), d(N)] MN-major B
  if (!ok) return CODA_ERR_LAUNCH;

  // 1. dgrad + RMSNorm backward + residual gradient + h2 + dgamma partials
  EpiRmsNormBackwardFull::Params p = {};
  p.h = reinterpret_cast<const __nv_bfloat16*>(h);
  p.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p.r = r;
  p.dh_out = reinterpret_cast<__nv_bfloat16*>(dh_out);
  p.qpart = dw.qpart;
  p.flags = dw.flags;
  p.epoch = dw.epoch;
  p.salt = salt;
  const SkParams skd =
      (pair && cp.nt == 0) ? dgrad_pieces(dw, M, d, N1, max_pairs, salt) : kNoSplitTail;
  if (skd.pieces > 0) units = max_pairs;
  p.dh_res = reinterpret_cast<const __nv_bfloat16*>(dh_res);
  p.h2_out = h2;
  p.gpart = gpart;
  cudaError_t e = pair ? launch(kPairDgradFull, 2 * units, kThreads, kPairDgradFullSmem, stream,
                                true, mDy, mW1, Mi, di, N1i, 1, p, skd, cp, tmo)
                       : launch(kDgradFull, units, kThreads, kDgradFullSmem, stream, true, mDy, mW1,
                                Mi, di, N1i, 1, p, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  // 2. dgamma = column sums of the partials
  e = launch(colsum_kernel, static_cast<int>(cdiv(d, 256)), 256, 0, stream, false,
             static_cast<const float*>(gpart), 4 * slabs, di, dgamma_out);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(1, stream);
  // 3. dW1 = h2^T dy   (K = tokens)
  EpiStoreF32::Params pw1 = {};
  pw1.out = dW1_out;
  const int mtw = static_cast<int>(cdiv(d, pair ? kPairBM : kBM));
  const int ntw1 = static_cast<int>(cdiv(N1, kBN));
  const int64_t nkw = cdiv(M, kBK);  // k-blocks of the weight gradients (K = tokens)
  const int npw1 = std::min(max_pairs, mtw * ntw1);
  const SkParams skw1 = plan_split_tail(skr, static_cast<int64_t>(mtw) * ntw1, npw1, nkw, salt);
  e = pair ? launch(kPairWgrad, 2 * npw1, kThreads, kPairWgradSmem, stream, skw1.epoch != nullptr,
                    mH2, mDyMN, di, N1i, Mi, kPairGroupM, pw1, skw1, kNoColPlan, tmo)
           : launch(kWgrad, std::min(sms, mtw * ntw1), kThreads, kWgradSmem, stream, false, mH2,
                    mDyMN, di, N1i, Mi, kGroupM, pw1, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(2, stream);
  // 4. dx = dh W0^T
  EpiRowScale::Params px = {};
  px.r = nullptr;
  px.y_out = reinterpret_cast<__nv_bfloat16*>(dx_out);
  const int mtx = static_cast<int>(cdiv(M, pair ? kPairBM : kBM));
  const int npx = std::min(max_pairs, mtx * nt);
  const SkParams skx =
      plan_split_tail(skr, static_cast<int64_t>(mtx) * nt, npx, cdiv(d, kBK), salt);
  e = pair ? launch(kPairXgrad, 2 * npx, kThreads, kPairXgradSmem, stream, skx.epoch != nullptr,
                    mDh, mW0, Mi, di, di, kPairGroupM, px, skx, kNoColPlan, tmo)
           : launch(kXgrad, std::min(sms, mtx * nt), kThreads, kXgradSmem, stream, false, mDh,
                    mW0, Mi, di, di, kGroupM, px, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(3, stream);
  // 5. dW0 = x^T dh   (K = tokens)
  EpiStoreF32::Params pw0 = {};
  pw0.out = dW0_out;
  const int npw0 = std::min(max_pairs, mtw * nt);
  const SkParams skw0 = plan_split_tail(skr, static_cast<int64_t>(mtw) * nt, npw0, nkw, salt);
  e = pair ? launch(kPairWgrad, 2 * npw0, kThreads, kPairWgradSmem, stream, skw0.epoch != nullptr,
                    mX, mDhMN, di, di, Mi, kPairGroupM, pw0, skw0, kNoColPlan, tmo)
           : launch(kWgrad, std::min(sms, mtw * nt), kThreads, kWgradSmem, stream, false, mX,
                    mDhMN, di, di, Mi, kGroupM, pw0, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(4, stream);
  return CODA_OK;
}

// [slot | s-partials | piece partials | piece flags]: launch 3 (the tile-local
// data gradient) may cut its last tiles into K pieces, like the data gradient.
size_t swiglu_spart_bytes(int64_t M, int64_t N1) {
  return align256(static_cast<size_t>(2 * cdiv(N1 / 2, kBN)) * M * 4);
}

size_t coda_bwd_swiglu_dgrad_workspace_bytes(int64_t M, int64_t d, int64_t N1, int64_t Dout) {
  if (check_common(M, d, N1) != CODA_OK || Dout <= 0 || M == 0) return 0;
  const int64_t ps = dgrad_piece_slots(M, d);
  return kSlotBytes + swiglu_spart_bytes(M, N1) +
         align256(static_cast<size_t>(ps) * 2 * kSkSlotFloats * 4) +
         align256(static_cast<size_t>(ps) * 2 * 8);
}

// The SwiGLU backward from the pre-activation saved as bf16 (y) or as an 8-bit
// checkpoint (y_q, y_s, with a_out optionally recomputed); the other form is null.
static coda_status_t swiglu_bwd_impl(const coda_bf16* dout, const coda_bf16* W2, const coda_bf16* y,
                                     const int8_t* y_q, const float* y_s, const coda_bf16* W1,
                                     const coda_bf16* h, const float* r, const coda_bf16* gamma,
                                     int64_t M, int64_t d, int64_t N1, int64_t Dout,
                                     coda_bf16* dy_out, float* s_out, coda_bf16* dh_out,
                                     coda_bf16* a_out, bool q8, void* workspace,
                                     size_t workspace_bytes, cudaStream_t stream) {
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (Dout <= 0) return CODA_ERR_INVALID_ARG;
  // bf16 rows of N1 / 2 values, or code rows of N1 / 2 bytes, on 16-byte boundaries
  if (N1 % (q8 ? 32 : 16) != 0 || Dout % 8 != 0 || Dout > (int64_t(1) << 31) - 256)
    return CODA_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return CODA_OK;
  if (!dout || !W2 || !(q8 ? y_q && y_s : y != nullptr) || !W1 || !h || !r || !gamma || !dy_out ||
      !s_out || !dh_out)
    return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dout, W2, y, y_q, y_s, W1, h, r, gamma, dy_out, s_out, dh_out, a_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  if (workspace == nullptr ||
      workspace_bytes < coda_bwd_swiglu_dgrad_workspace_bytes(M, d, N1, Dout))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  st = device_setup(&sms, &max_pairs);
  if (st != CODA_OK) return st;
  const bool pair = g_mma_mode.load() == 1;
  const int64_t half = N1 / 2;
  const int Mi = static_cast<int>(M), di = static_cast<int>(d), N1i = static_cast<int>(N1);
  const int halfi = static_cast<int>(half), Douti = static_cast<int>(Dout);
  const uint64_t tmo = g_timeout_ns.load();

  CUtensorMap mA0, mB0, mA1, mB1;
  const uint32_t bbox = pair ? 128 : kBN;
  bool ok = tmap_2d(&mA0, dout, Dout, M, kBK, kBM);   // dout [M, Dout]       K-major (K = Dout)
  ok &= tmap_2d(&mB0, W2, Dout, half, kBK, bbox);     // W2 [half(N), Dout(K)] K-major
  ok &= tmap_2d(&mA1, dy_out, N1, M, kBK, kBM);       // dy [M, N1]           K-major (K = N1)
  ok &= tmap_2d(&mB1, W1, N1, d, kBK, bbox);          // W1 [d(N), N1(K)]      K-major
  if (!ok) return CODA_ERR_LAUNCH;

  const int nts = static_cast<int>(cdiv(half, kBN));
  const int ntd = static_cast<int>(cdiv(d, kBN));
  const int mt = static_cast<int>(cdiv(M, kBM));
  const int mtp = static_cast<int>(cdiv(M, kPairBM));

  // 1. down-projection data gradient with the SwiGLU backward + partial s
  EpiSwiGLUBackward::Params p0 = {};
  p0.y = reinterpret_cast<const __nv_bfloat16*>(y);
  p0.dy_out = reinterpret_cast<__nv_bfloat16*>(dy_out);
  p0.spart = reinterpret_cast<float*>(static_cast<char*>(workspace) + kSlotBytes);
  EpiSwiGLUBackwardQ8::Params p0q = {};
  p0q.y_q = reinterpret_cast<const uint8_t*>(y_q);
  p0q.y_s = y_s;
  p0q.nb = static_cast<int>(cdiv(N1, kQ8Block));
  p0q.dy_out = p0.dy_out;
  p0q.a_out = reinterpret_cast<__nv_bfloat16*>(a_out);
  p0q.spart = p0.spart;
  cudaError_t e;
  if (q8)
    e = pair ? launch(kPairSwigluBwdQ8, 2 * std::min(max_pairs, mtp * nts), kThreads,
                      kPairSwigluBwdQ8Smem, stream, false, mA0, mB0, Mi, halfi, Douti, kPairGroupM,
                      p0q, kNoSplitTail, kNoColPlan, tmo)
             : launch(kSwigluBwdQ8, std::min(sms, mt * nts), kThreads, kSwigluBwdQ8Smem, stream,
                      false, mA0, mB0, Mi, halfi, Douti, kGroupM, p0q, tmo);
  else
    e = pair ? launch(kPairSwigluBwd, 2 * std::min(max_pairs, mtp * nts), kThreads,
                      kPairSwigluBwdSmem, stream, false, mA0, mB0, Mi, halfi, Douti, kPairGroupM,
                      p0, kNoSplitTail, kNoColPlan, tmo)
             : launch(kSwigluBwd, std::min(sms, mt * nts), kThreads, kSwigluBwdSmem, stream, false,
                      mA0, mB0, Mi, halfi, Douti, kGroupM, p0, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  // 2. light auxiliary reduction of the statistic
  e = launch(rowsum_kernel, static_cast<int>(cdiv(M, 256)), 256, 0, stream, false,
             static_cast<const float*>(p0.spart), 2 * nts, Mi, s_out);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(1, stream);
  // 3. RMSNorm-branch data gradient, tile-local with s given; its last tiles may
  // be cut into K pieces (any tiles: no row statistic ties them together)
  EpiRmsNormBackwardGivenS::Params p1 = {};
  p1.h = reinterpret_cast<const __nv_bfloat16*>(h);
  p1.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p1.r = r;
  p1.s = s_out;
  p1.dh_out = reinterpret_cast<__nv_bfloat16*>(dh_out);
  SkParams sk3 = kNoSplitTail;
  if (pair && g_dgrad_pieces.load() != 0) {
    const int64_t pslots = dgrad_piece_slots(M, d);
    const PiecePlan pp = piece_plan_for(M, d, N1, max_pairs, true);
    if (pp.pieces > 0) {
      char* pbase = static_cast<char*>(workspace) + kSlotBytes + swiglu_spart_bytes(M, N1);
      sk3.dp_tiles = pp.dp_tiles;
      sk3.part = reinterpret_cast<float*>(pbase);
      sk3.flags = reinterpret_cast<uint64_t*>(
          pbase + align256(static_cast<size_t>(pslots) * 2 * kSkSlotFloats * 4));
      sk3.epoch = static_cast<uint64_t*>(workspace);
      sk3.slots = static_cast<int>(pslots);
      sk3.salt = next_salt();
      sk3.pieces = pp.pieces;
      sk3.lvl_first = pp.lvl_first;
      sk3.lvl = pp.lvl;
    }
  }
  const int units3 = sk3.pieces > 0 ? max_pairs : std::min(max_pairs, mtp * ntd);
  e = pair ? launch(kPairDgradGivenS, 2 * units3, kThreads, kPairDgradGivenSSmem, stream,
                    sk3.pieces > 0, mA1, mB1, Mi, di, N1i, kPairGroupM, p1, sk3, kNoColPlan, tmo)
           : launch(kDgradGivenS, std::min(sms, mt * ntd), kThreads, kDgradGivenSSmem, stream,
                    false, mA1, mB1, Mi, di, N1i, kGroupM, p1, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(2, stream);
  return CODA_OK;
}

coda_status_t coda_bwd_swiglu_dgrad(const coda_bf16* dout, const coda_bf16* W2, const coda_bf16* y,
                                    const coda_bf16* W1, const coda_bf16* h, const float* r,
                                    const coda_bf16* gamma, int64_t M, int64_t d, int64_t N1,
                                    int64_t Dout, coda_bf16* dy_out, float* s_out,
                                    coda_bf16* dh_out, void* workspace, size_t workspace_bytes,
                                    cudaStream_t stream) {
  return swiglu_bwd_impl(dout, W2, y, nullptr, nullptr, W1, h, r, gamma, M, d, N1, Dout, dy_out,
                         s_out, dh_out, nullptr, false, workspace, workspace_bytes, stream);
}

coda_status_t coda_bwd_swiglu_dgrad_q8(const coda_bf16* dout, const coda_bf16* W2,
                                       const int8_t* y_q, const float* y_s, const coda_bf16* W1,
                                       const coda_bf16* h, const float* r, const coda_bf16* gamma,
                                       int64_t M, int64_t d, int64_t N1, int64_t Dout,
                                       coda_bf16* dy_out, float* s_out, coda_bf16* dh_out,
                                       coda_bf16* a_out, void* workspace, size_t workspace_bytes,
                                       cudaStream_t stream) {
  return swiglu_bwd_impl(dout, W2, nullptr, y_q, y_s, W1, h, r, gamma, M, d, N1, Dout, dy_out,
                         s_out, dh_out, a_out, true, workspace, workspace_bytes, stream);
}

coda_status_t coda_quant_q8(const coda_bf16* x, int64_t M, int64_t n, int block, int8_t* q_out,
                            float* s_out, cudaStream_t stream) {
  coda_status_t st = check_rows(M, n);
  if (st != CODA_OK) return st;
  if (block != 0 && block != kQ8Block) return CODA_ERR_INVALID_ARG;
  if (M == 0) return CODA_OK;
  if (!x || !q_out || !s_out) return CODA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q_out) || !aligned16(s_out)) return CODA_ERR_MISALIGNED;
  dim3 grid;
  if (!q8_block_grid(M, n, kQ8QuantLanes, &grid)) return CODA_ERR_UNSUPPORTED_SHAPE;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  cudaError_t e;
  if (block == 0) {
    RowQ8Params p = {};
    p.x = reinterpret_cast<const __nv_bfloat16*>(x);
    p.q_out = reinterpret_cast<uint8_t*>(q_out);
    p.s_out = s_out;
    p.M = static_cast<int>(M);
    p.d = static_cast<int>(n);
    e = launch_row_q8<false, false, false>(p, sms, stream);
  } else {
    e = launch(block_q8_kernel, grid, 256, 0, stream, false,
               reinterpret_cast<const __nv_bfloat16*>(x), reinterpret_cast<uint8_t*>(q_out), s_out,
               static_cast<int>(M), static_cast<int>(n));
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

coda_status_t coda_dequant_q8(const int8_t* q, const float* s, int64_t M, int64_t n, int block,
                              coda_bf16* x_out, cudaStream_t stream) {
  coda_status_t st = check_rows(M, n);
  if (st != CODA_OK) return st;
  if (block != 0 && block != kQ8Block) return CODA_ERR_INVALID_ARG;
  if (M == 0) return CODA_OK;
  if (!q || !s || !x_out) return CODA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(s) || !aligned16(x_out)) return CODA_ERR_MISALIGNED;
  dim3 grid;
  if (!q8_block_grid(M, n, kQ8DequantLanes, &grid)) return CODA_ERR_UNSUPPORTED_SHAPE;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  const uint8_t* qb = reinterpret_cast<const uint8_t*>(q);
  __nv_bfloat16* xb = reinterpret_cast<__nv_bfloat16*>(x_out);
  const cudaError_t e = launch(block == 0 ? &dequant_q8_kernel<true> : &dequant_q8_kernel<false>,
                               grid, 256, 0, stream, false, qb, s, xb, static_cast<int>(M),
                               static_cast<int>(n));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

coda_status_t coda_add_rmsnorm_q8(const coda_bf16* x, const coda_bf16* z, const coda_bf16* gamma,
                                  float eps, int64_t M, int64_t d, coda_bf16* h_out, int8_t* q_out,
                                  float* s_out, cudaStream_t stream) {
  coda_status_t st = check_rows(M, d);
  if (st != CODA_OK) return st;
  if (M == 0) return CODA_OK;
  if (!x || !gamma || !q_out || !s_out) return CODA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {x, z, gamma, h_out, q_out, s_out};  // z and h_out may be null
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  RowQ8Params p = {};
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.z = reinterpret_cast<const __nv_bfloat16*>(z);
  p.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p.h_out = reinterpret_cast<__nv_bfloat16*>(h_out);
  p.q_out = reinterpret_cast<uint8_t*>(q_out);
  p.s_out = s_out;
  p.eps = eps;
  p.M = static_cast<int>(M);
  p.d = static_cast<int>(d);
  const cudaError_t e = z ? (h_out ? launch_row_q8<true, true, true>(p, sms, stream)
                                   : launch_row_q8<true, true, false>(p, sms, stream))
                          : (h_out ? launch_row_q8<true, false, true>(p, sms, stream)
                                   : launch_row_q8<true, false, false>(p, sms, stream));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

// Nothing up to kMidSure tokens; then
// [slot | a as bf16 integers | W as bf16 integers | split-tail region]
size_t coda_matmul_q8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (check_product(M, K, N) != CODA_OK || M <= kMidSure) return 0;
  return kSlotBytes + align256(static_cast<size_t>(M) * K * 2) +
         align256(static_cast<size_t>(K) * N * 2) + sk_region_bytes(cdiv(M, kPairBM) * cdiv(N, kBN));
}

int coda_matmul_q8_plan(int64_t M, int64_t K, int64_t N, int sms, int pairs, const int32_t* clusters,
                        int32_t* plan) {
  if (plan == nullptr || clusters == nullptr || check_product(M, K, N) != CODA_OK || M == 0 ||
      sms < 1 || pairs < 0)
    return -1;
  int fit[2][3];
  for (int i = 0; i < 3; ++i) {
    if (clusters[i] < 0) return -1;
    fit[0][i] = clusters[i];
    fit[1][i] = 2 * clusters[i];
  }
  const ProductPlan p = plan_product(M, K, N, sms, pairs, fit);
  plan[0] = p.split;
  plan[1] = p.form == kFormMid ? p.mid.tokens : 0;
  plan[2] = p.form == kFormMid && p.mid.narrow;
  return static_cast<int>(p.form);
}

coda_status_t coda_matmul_q8(const int8_t* a_q, const float* a_s, const int8_t* W_q,
                             const float* w_s, const coda_bf16* z, int64_t M, int64_t K, int64_t N,
                             coda_bf16* y_out, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  coda_status_t st = check_product(M, K, N);
  if (st != CODA_OK) return st;
  if (M == 0) return CODA_OK;
  if (!a_q || !a_s || !W_q || !w_s || !y_out) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {a_q, a_s, W_q, w_s, z, y_out};  // z may be null
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  const size_t need = coda_matmul_q8_workspace_bytes(M, K, N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned16(workspace)) return CODA_ERR_MISALIGNED;
  int sms = 0, max_pairs = 0;
  const int (*clusters)[3] = nullptr;
  st = device_setup(&sms, &max_pairs, nullptr, &clusters);
  if (st != CODA_OK) return st;
  const bool pair = g_mma_mode.load() == 1;
  const uint64_t tmo = g_timeout_ns.load();
  const int Mi = static_cast<int>(M), Ki = static_cast<int>(K), Ni = static_cast<int>(N);

  const ProductPlan plan = plan_product(M, K, N, sms, max_pairs, clusters);
  if (plan.form == kFormNone) return CODA_ERR_LAUNCH;

  if (plan.form == kFormSmall) {
    SmallQ8Params sp = {};
    sp.a_s = a_s;
    sp.w_s = w_s;
    sp.z = reinterpret_cast<const __nv_bfloat16*>(z);
    sp.y = reinterpret_cast<__nv_bfloat16*>(y_out);
    sp.M = Mi;
    sp.K = Ki;
    sp.N = Ni;
    if (launch_product_small(sp, reinterpret_cast<const uint8_t*>(a_q),
                             reinterpret_cast<const uint8_t*>(W_q), plan.split, stream) != cudaSuccess) {
      cudaGetLastError();
      return CODA_ERR_LAUNCH;
    }
    after_launch(0, stream);
    return CODA_OK;
  }
  if (plan.form == kFormMid) {
    MidQ8Params mp = {};
    mp.a_s = a_s;
    mp.w_s = w_s;
    mp.z = reinterpret_cast<const __nv_bfloat16*>(z);
    mp.y = reinterpret_cast<__nv_bfloat16*>(y_out);
    mp.M = Mi;
    mp.K = Ki;
    mp.N = Ni;
    if (launch_product_mid(mp, reinterpret_cast<const uint8_t*>(a_q),
                           reinterpret_cast<const uint8_t*>(W_q), plan.mid, stream) != cudaSuccess) {
      cudaGetLastError();
      return CODA_ERR_LAUNCH;
    }
    return CODA_OK;
  }
  char* wsb = static_cast<char*>(workspace);
  __nv_bfloat16* a = reinterpret_cast<__nv_bfloat16*>(wsb + kSlotBytes);
  __nv_bfloat16* W =
      reinterpret_cast<__nv_bfloat16*>(wsb + kSlotBytes + align256(static_cast<size_t>(M) * K * 2));
  const int64_t mtp = cdiv(M, kPairBM), nt = cdiv(N, kBN);
  const SkRegion skr = sk_region(reinterpret_cast<char*>(W) + align256(static_cast<size_t>(K) * N * 2),
                                 mtp * nt, wsb);
  CUtensorMap mA, mB;
  bool ok = tmap_2d(&mA, a, K, M, kBK, kBM);  // [M, K] K-major
  ok &= tmap_2d(&mB, W, N, K, 64, kBK);       // [K, N] MN-major
  if (!ok) return CODA_ERR_LAUNCH;

  const size_t na = static_cast<size_t>(M) * K / 16, nw = static_cast<size_t>(K) * N / 16;
  cudaError_t e = launch(q8_to_bf16_kernel, static_cast<int>(cdiv(na, 256)), 256, 0, stream, false,
                         reinterpret_cast<const uint8_t*>(a_q), a, na);
  if (e == cudaSuccess) {
    after_launch(0, stream);
    e = launch(q8_to_bf16_kernel, static_cast<int>(cdiv(nw, 256)), 256, 0, stream, false,
               reinterpret_cast<const uint8_t*>(W_q), W, nw);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(1, stream);
  EpiTokenChannelScale::Params p = {};
  p.a_s = a_s;
  p.w_s = w_s;
  p.z = reinterpret_cast<const __nv_bfloat16*>(z);
  p.y_out = reinterpret_cast<__nv_bfloat16*>(y_out);
  const int units = static_cast<int>(std::min<int64_t>(max_pairs, mtp * nt));
  const SkParams sk = plan_split_tail(skr, mtp * nt, units, cdiv(K, kBK), next_salt());
  e = pair ? launch(kPairProductQ8, 2 * units, kThreads, kPairProductQ8Smem, stream,
                    sk.epoch != nullptr, mA, mB, Mi, Ni, Ki, kPairGroupM, p, sk, kNoColPlan, tmo)
           : launch(kProductQ8, static_cast<int>(std::min<int64_t>(sms, cdiv(M, kBM) * nt)), kThreads,
                    kProductQ8Smem, stream, false, mA, mB, Mi, Ni, Ki, kGroupM, p, tmo);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(2, stream);
  return CODA_OK;
}

coda_status_t coda_cache_write_q8(const coda_bf16* y, int8_t* k_q, float* k_s, int8_t* v_q, float* v_s,
                                  int64_t pages, int64_t Hk, int64_t page, int64_t D, const int32_t* cu,
                                  const int32_t* lens, const int32_t* table, int64_t B, int64_t width,
                                  int64_t T, int64_t Hq, const double* inv_freq, const int32_t* axis,
                                  int64_t half, const int32_t* pos, int64_t axes, int pairs,
                                  coda_bf16* q_out, cudaStream_t stream) {
  CacheWriteParams p = {};
  coda_status_t st = check_cache(k_q, k_s, v_q, v_s, pages, Hq, Hk, page, D, cu, lens, table, B, width, T,
                                 &p.cache, &p.batch);
  if (st != CODA_OK) return st;
  RopeQ8 r;
  st = rope_of(inv_freq, axis, half, pos, axes, pairs, D, &r);
  if (st != CODA_OK) return st;
  if (T == 0 || B == 0) return CODA_OK;
  if (!y || !q_out) return CODA_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(q_out)) return CODA_ERR_MISALIGNED;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  p.y = reinterpret_cast<const __nv_bfloat16*>(y);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.Hq = static_cast<int>(Hq);
  const cudaError_t e = D == 64 ? launch_cache_write<64>(p, r, sms, stream)
                                : launch_cache_write<128>(p, r, sms, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

coda_status_t coda_cache_read_q8(const int8_t* k_q, const float* k_s, const int8_t* v_q, const float* v_s,
                                 int64_t pages, int64_t Hk, int64_t page, int64_t D, const int32_t* cu,
                                 const int32_t* lens, const int32_t* table, int64_t B, int64_t width,
                                 int64_t T, coda_bf16* k_out, coda_bf16* v_out, cudaStream_t stream) {
  CacheReadParams p = {};
  coda_status_t st = check_cache(k_q, k_s, v_q, v_s, pages, Hk, Hk, page, D, cu, lens, table, B, width, T,
                                 &p.cache, &p.batch);
  if (st != CODA_OK) return st;
  if (T == 0 || B == 0) return CODA_OK;
  if (!k_out || !v_out) return CODA_ERR_INVALID_ARG;
  if (!aligned16(k_out) || !aligned16(v_out)) return CODA_ERR_MISALIGNED;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  p.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  p.v_out = reinterpret_cast<__nv_bfloat16*>(v_out);
  const cudaError_t e = D == 64 ? launch_cache_read<64>(p, sms, stream) : launch_cache_read<128>(p, sms, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  after_launch(0, stream);
  return CODA_OK;
}

size_t coda_attn_q8_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hk, int64_t D) {
  if (check_heads(T, B, Hq, Hk, D) != CODA_OK || T == 0 || B == 0) return 0;
  const int64_t rows = T * (Hq / Hk);
  return kSlotBytes + attn_ws_bytes(kFewRows, rows, D) + (rows > kFewMost ? attn_ws_bytes(kTileRows, kTileRows, D) : 0);
}

coda_status_t coda_attn_q8(const coda_bf16* q, const int8_t* k_q, const float* k_s, const int8_t* v_q,
                           const float* v_s, int64_t pages, int64_t Hk, int64_t page, int64_t D,
                           const int32_t* cu, const int32_t* lens, const int32_t* table, int64_t B,
                           int64_t width, int64_t T, int64_t Hq, float scale, int64_t most,
                           coda_bf16* o_out, float* lse_out, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  AttnQ8Params p = {};
  coda_status_t st = check_cache(k_q, k_s, v_q, v_s, pages, Hq, Hk, page, D, cu, lens, table, B, width, T,
                                 &p.cache, &p.batch);
  if (st != CODA_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f || most < 0) return CODA_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return CODA_OK;
  if (!q || !o_out) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, o_out, lse_out, workspace};  // lse_out may be null
  for (const void* ptr : ptrs)
    if (!aligned16(ptr)) return CODA_ERR_MISALIGNED;
  if (workspace == nullptr || workspace_bytes < coda_attn_q8_workspace_bytes(T, B, Hq, Hk, D))
    return CODA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  st = device_setup(&sms);
  if (st != CODA_OK) return st;
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.o = reinterpret_cast<__nv_bfloat16*>(o_out);
  p.lse = lse_out;
  p.Hq = static_cast<int>(Hq);
  p.group = static_cast<int>(Hq / Hk);
  int power = 0;
  p.scale_part = 2.0f * std::frexp(scale, &power) * 1.44269504088896f;
  p.scale_power = std::ldexp(1.0f, power - 1);
  const int blocks = std::min(sms, kAttnMaxBlocks);
  char* const wsb = static_cast<char*>(workspace) + kSlotBytes;
  // the most packed rows that a sequence may have
  const int64_t rows = std::min(most > 0 ? most : T, T) * p.group;
  const cudaError_t e = D == 64 ? launch_attn<64>(p, wsb, rows, most > 0, blocks, stream)
                                : launch_attn<128>(p, wsb, rows, most > 0, blocks, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  return CODA_OK;
}

coda_status_t coda_get_device_status(cudaStream_t stream, uint32_t* detail) {
  if (detail) *detail = 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_NO_DEVICE;
  }
  if (cudaStreamSynchronize(stream) != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, coda::g_coda_status, sizeof(v)) != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  if (v != 0) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(coda::g_coda_status, &zero, sizeof(zero)) != cudaSuccess) {
      cudaGetLastError();
      return CODA_ERR_LAUNCH;
    }
  }
  if (detail) *detail = v;
  if (v == 0) return CODA_OK;
  return (v & 0x200u) ? CODA_ERR_DEVICE_BOUNDS : CODA_ERR_DEVICE_TIMEOUT;
}

void coda_set_launch_events(cudaEvent_t* events, int n) {
  g_launch_events = (n > 0) ? events : nullptr;
  g_launch_events_n = (n > 0) ? n : 0;
}

coda_status_t coda_set_mma_mode(int mode) {
  if (mode != 0 && mode != 1) return CODA_ERR_INVALID_ARG;
  g_mma_mode.store(mode);
  return CODA_OK;
}

int coda_get_mma_mode(void) { return g_mma_mode.load(); }

coda_status_t coda_set_split_tail(int enable) {
  if (enable != 0 && enable != 1) return CODA_ERR_INVALID_ARG;
  g_split_tail.store(enable);
  return CODA_OK;
}

coda_status_t coda_set_col_plan(int enable) {
  if (enable < 0 || enable > 2) return CODA_ERR_INVALID_ARG;
  g_col_plan.store(enable);
  return CODA_OK;
}

coda_status_t coda_set_serpentine_k(int enable) {
  if (enable != 0 && enable != 1) return CODA_ERR_INVALID_ARG;
  g_dgrad_kserp.store(enable);
  return CODA_OK;
}

int coda_get_serpentine_k(void) { return g_dgrad_kserp.load(); }

coda_status_t coda_set_dgrad_pieces(int enable) {
  if (enable != 0 && enable != 1) return CODA_ERR_INVALID_ARG;
  g_dgrad_pieces.store(enable);
  return CODA_OK;
}

int coda_get_dgrad_pieces(void) { return g_dgrad_pieces.load(); }

int coda_dgrad_piece_plan(int64_t M, int64_t d, int64_t N1, int npairs, int tile_local,
                          int32_t* plan) {
  if (plan == nullptr || npairs < 1 || check_common(M, d, N1) != CODA_OK || M == 0) return -1;
  const PiecePlan pp = piece_plan_for(M, d, N1, npairs, tile_local != 0);
  plan[0] = pp.dp_tiles;
  plan[1] = pp.pieces;
  plan[2] = pp.lvl_first;
  plan[3] = pp.lvl;
  return pp.pieces > 0 ? 1 : 0;
}

coda_status_t coda_set_fold_rowreduce(int enable) {
  if (enable != 0 && enable != 1) return CODA_ERR_INVALID_ARG;
  g_fold_rowreduce.store(enable);
  return CODA_OK;
}

void coda_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns == 0 ? 1 : ns); }

const char* coda_status_string(coda_status_t s) {
  switch (s) {
    case CODA_OK: return "CODA_OK";
    case CODA_ERR_INVALID_ARG: return "CODA_ERR_INVALID_ARG";
    case CODA_ERR_UNSUPPORTED_SHAPE: return "CODA_ERR_UNSUPPORTED_SHAPE";
    case CODA_ERR_MISALIGNED: return "CODA_ERR_MISALIGNED";
    case CODA_ERR_WORKSPACE_TOO_SMALL: return "CODA_ERR_WORKSPACE_TOO_SMALL";
    case CODA_ERR_LAUNCH: return "CODA_ERR_LAUNCH";
    case CODA_ERR_DEVICE_TIMEOUT: return "CODA_ERR_DEVICE_TIMEOUT";
    case CODA_ERR_NO_DEVICE: return "CODA_ERR_NO_DEVICE";
    case CODA_ERR_UNSUPPORTED_DEVICE: return "CODA_ERR_UNSUPPORTED_DEVICE";
    case CODA_ERR_DEVICE_BOUNDS: return "CODA_ERR_DEVICE_BOUNDS";
  }
  return "CODA_ERR_UNKNOWN";
}

coda_status_t coda_watchdog_selftest(uint64_t timeout_ns, cudaStream_t stream) {
  int sms = 0;
  coda_status_t st = device_setup(&sms);
  if (st != CODA_OK) return st;
  cudaError_t e = launch(coda::watchdog_selftest_kernel, 1, 32, 0, stream, false, timeout_ns);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  return CODA_OK;
}

}  // extern "C"

extern "C" coda_status_t coda_bwd_dgrad_noalloc(const coda_bf16* dy, const coda_bf16* W1,
                                                const coda_bf16* h, const float* r,
                                                const coda_bf16* gamma, int64_t M, int64_t d,
                                                int64_t N1, coda_bf16* dh_out,
                                                cudaStream_t stream) {
  coda_status_t st = check_common(M, d, N1);
  if (st != CODA_OK) return st;
  if (M == 0) return CODA_OK;
  if (!dy || !W1 || !h || !r || !gamma || !dh_out) return CODA_ERR_INVALID_ARG;
  const void* ptrs[] = {dy, W1, h, r, gamma, dh_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CODA_ERR_MISALIGNED;
  const int64_t mt64 = cdiv(M, kBM), nt64 = cdiv(d, kBN);
  if (2 * static_cast<uint64_t>(nt64) * static_cast<uint64_t>(M) > kNoAllocPartials ||
      static_cast<uint64_t>(mt64) * static_cast<uint64_t>(nt64) > kNoAllocFlags)
    return CODA_ERR_UNSUPPORTED_SHAPE;  // larger than the static scratch
  int sms = 0;
  void* scratch = nullptr;
  st = device_setup(&sms, nullptr, &scratch);
  if (st != CODA_OK) return st;

  const int mt = static_cast<int>(mt64);
  const int nt = static_cast<int>(nt64);
  const int grid = std::min(sms, mt * nt);
  if (nt > grid) return CODA_ERR_UNSUPPORTED_SHAPE;

  CUtensorMap mA, mB;
  bool ok = tmap_2d(&mA, dy, N1, M, kBK, kBM);
  ok &= tmap_2d(&mB, W1, N1, d, kBK, kBN);
  if (!ok) return CODA_ERR_LAUNCH;

  EpiRmsNormBackward::Params p = {};
  p.h = reinterpret_cast<const __nv_bfloat16*>(h);
  p.gamma = reinterpret_cast<const __nv_bfloat16*>(gamma);
  p.r = r;
  p.dh_out = reinterpret_cast<__nv_bfloat16*>(dh_out);
  p.qpart = reinterpret_cast<float*>(scratch);
  p.flags = reinterpret_cast<uint64_t*>(static_cast<unsigned char*>(scratch) + kNoAllocFlagOffset);
  p.epoch = reinterpret_cast<uint64_t*>(static_cast<unsigned char*>(scratch) + kNoAllocEpochOffset);
  p.salt = next_salt();
  cudaError_t e = launch(kDgrad, grid, kThreads, kDgradSmem, stream, true, mA, mB,
                         static_cast<int>(M), static_cast<int>(d), static_cast<int>(N1), 1, p,
                         g_timeout_ns.load());
  if (e != cudaSuccess) {
    cudaGetLastError();
    return CODA_ERR_LAUNCH;
  }
  return CODA_OK;
}
