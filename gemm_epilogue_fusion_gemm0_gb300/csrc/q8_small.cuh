// q8_small.cuh -- the INT8 product for few tokens: the weights' bytes at the rate of HBM.
//
//   y[m, n] = a_s[m] w_s[n] sum_k a[m, k] W[k, n] (+ z),   M <= 32 tokens, W [K, N] INT8
//
// Every byte of W is used for at most 32 tokens, so the kernel is bound by reading W once
// and its design is about keeping loads in flight: each warp owns 128 channels and a
// private ring of steps of 32 rows of W (4 KB) and of the tokens' 32 codes, filled by
// TMA and guarded by one mbarrier per stage; no barrier is shared between warps in the
// loop.  (With W loaded straight to registers, two steps ahead, 8 warps hold at most
// 64 KB in flight and 16 to 32 tokens ran at 37 to 53 % of HBM's rate.)
//
// The products run as mma.sync.m16n8k16 on fp16, W^T being the 16 x 16 operand and the
// tokens the 8 columns.  tcgen05 has no INT8 form on sm_103a and mma.sync's INT8 form
// measured 252 multiply-adds per cycle and SM there, fp16 1020: codes are exact in fp16, and a
// step of 4 KB, 180 cycles of an SM's share of HBM, holds 32 cycles of fp16 instructions
// per 8 tokens.  The tensor memory form would need W in shared memory in 16 bits, which
// costs more shared-memory traffic than a byte's share of time.
//
// A code becomes fp16 by its bits: 0x6400 | (code + 128) is 1024 + 128 + code, and a
// packed subtraction of 1152 leaves the code exactly: 1.5 instructions per code.
//
// Rows and columns of an instruction may be dealt freely as long as both operands agree:
//   row g      of tile j = channel 16 c(g) + 2 j       (g = lane / 4, t = lane % 4)
//   row g + 8  of tile j = channel 16 c(g) + 2 j + 1
//   k 2t, 2t+1, 2t+8, 2t+9 of instruction q = rows 4 i + t of the step, i = 4 q .. 4 q + 3
// so a thread's 16-byte reads of W are its own operands for tiles j = 0..7 and its sums for
// tiles 2i, 2i + 1 are four neighbouring channels.  With the 128-byte swizzle the 16-byte
// group c of row r sits at c ^ (r % 8); c(g) = g / 2 + 4 (g % 2) lets the eight lanes that
// read together (two g, four t) touch all eight groups: no bank conflicts.
//
// K is split over the block's 8 warps and over a cluster of up to 8 blocks.  The fp32
// sums of a block's warps meet in shared memory once, at the end, then each block adds the
// cluster's parts of its share of the outputs through distributed shared memory, all in a
// fixed order (bit-reproducible).
#pragma once

#include "q8.cuh"

namespace coda {

constexpr int kSmallChannels = 128;  // channels per block
constexpr int kSmallWarps = 8;
constexpr int kSmallStep = 32;       // rows of W per step of a warp
constexpr int kSmallMaxTokens = 32;

struct SmallQ8Params {
  const float* a_s;        // [M]
  const float* w_s;        // [N]
  const __nv_bfloat16* z;  // [M, N] or null
  __nv_bfloat16* y;        // [M, N]
  int M, K, N;
};

// 0x64uu 0x64uu (u = code + 128) -> the two codes in fp16
__device__ __forceinline__ uint32_t q8_less_1152(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0x64806480u));
  return r;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Ring stages per warp: as many as leave room for two blocks per SM up to 16 tokens (their
// sums fit half the registers), or one block beyond.
template <int kGroups>
constexpr int kSmallStages = kGroups <= 2 ? 3 : 5;
constexpr uint32_t kSmallWBytes = kSmallStep * kSmallChannels;  // one stage of W: 4 KB

// shared memory: W stages [warp][stage], token stages [warp][stage], barriers, the abort
// flag; the warps' sums (one float4 per warp, tile, token group and lane) take the W
// stages' place at the end
template <int kGroups>
struct SmallSmem {
  static constexpr uint32_t kXBytes = 8u * kGroups * kSmallStep;
  static constexpr uint32_t kX = kSmallWarps * kSmallStages<kGroups> * kSmallWBytes;
  static constexpr uint32_t kBar = kX + kSmallWarps * kSmallStages<kGroups> * kXBytes;
  static constexpr uint32_t kAbort = kBar + 8u * kSmallWarps * kSmallStages<kGroups>;
  static constexpr uint32_t kBytes = kAbort + 16 + 1024;  // 1 KB alignment slack
  static_assert(kSmallWarps * 8u * kGroups * 32u * 16u <= kX, "the sums overflow the ring");
  static_assert(kBytes <= (kGroups <= 2 ? 115712u : 232448u), "blocks per SM");
};

// kGroups: groups of 8 tokens (1, 2 or 4)
template <int kGroups>
__global__ void __launch_bounds__(32 * kSmallWarps, kGroups <= 2 ? 2 : 1)
    product_q8_small_kernel(const __grid_constant__ CUtensorMap tmW,
                            const __grid_constant__ CUtensorMap tmA, const SmallQ8Params p,
                            int split, uint64_t timeout_ns) {
  using Smem = SmallSmem<kGroups>;
  constexpr int kStagesS = kSmallStages<kGroups>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  // (from one lane: known to be the same in the whole warp, which keeps a copy's operands uniform)
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const bool issuer = elect_one();
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int n0 = static_cast<int>(blockIdx.x) / split * kSmallChannels;
  const uint32_t sW = base + static_cast<uint32_t>(warp) * kStagesS * kSmallWBytes;
  const uint32_t sX = base + Smem::kX + static_cast<uint32_t>(warp) * kStagesS * Smem::kXBytes;
  const uint32_t bar = base + Smem::kBar + 8u * warp * kStagesS;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Smem::kAbort);
  const WaitCtl wc{timeout_ns, &g_coda_status, abort_flag};
  if (threadIdx.x == 0) *abort_flag = 0u;
  if (lane == 0) {
    for (int s = 0; s < kStagesS; ++s) mbar_init(bar + 8u * s, 1);
    fence_mbar_init();
    if (warp == 0) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmA);
    }
  }
  __syncthreads();
  griddep_launch_dependents();

  // steps of this warp: first, first + stride, ... below nstep; rows past K and channels
  // past N read as zeros
  const int nstep = (p.K + kSmallStep - 1) / kSmallStep;
  const int first = warp * split + rank, stride = kSmallWarps * split;
  const int count = first < nstep ? (nstep - 1 - first) / stride + 1 : 0;
  const auto issue = [&](int i) {  // one lane: the i-th step of this warp into its stage
    const int k0 = (first + i * stride) * kSmallStep;
    const uint32_t st = static_cast<uint32_t>(i % kStagesS);
    if (!checked(tma_start_ok(n0, k0, p.N, p.K, 1), kChkTmaB) ||
        !checked(tma_start_ok(k0, 0, p.K, p.M, 1), kChkTmaA)) {
      *wc.abort_flag = 1u;  // the waits below give up
      return;
    }
    mbar_arrive_expect_tx(bar + 8u * st, kSmallWBytes + Smem::kXBytes);
    tma_load_2d(sW + st * kSmallWBytes, &tmW, bar + 8u * st, n0, k0);
    tma_load_2d(sX + st * Smem::kXBytes, &tmA, bar + 8u * st, k0, 0);
  };
  int issued = min(count, kStagesS);
  // While the kernel before this one finishes, the ring's first boxes of W are brought
  // into L2 (the point of coherence: nothing is read into this kernel yet).
  if (issuer)
    for (int i = 0; i < issued; ++i)
      tma_prefetch_l2_2d(&tmW, n0, (first + i * stride) * kSmallStep);
  griddep_wait();
  if (issuer)
    for (int i = 0; i < issued; ++i) issue(i);

  float acc[8][kGroups][4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < kGroups; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][c][e] = 0.f;

  const uint32_t col = static_cast<uint32_t>((g >> 1) | ((g & 1) << 2));  // c(g)
  // byte t of two words into bytes 0 and 2 (the others are masked away)
  const uint32_t sel_x = static_cast<uint32_t>(t) | static_cast<uint32_t>(4 + t) << 8;
  int done = 0;
  for (; done < count; ++done) {
    const uint32_t st = static_cast<uint32_t>(done % kStagesS);
    const uint32_t parity = static_cast<uint32_t>(done / kStagesS) & 1u;
    if (!__all_sync(0xffffffffu, bounded_wait(bar + 8u * st, parity, wc, kSiteMmaFull))) break;
    uint4 w[8], x[kGroups][2];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = 4 * i + static_cast<uint32_t>(t);
      w[i] = ld_shared_v4(sW + st * kSmallWBytes + 128u * r + 16u * (col ^ (r & 7u)));
    }
#pragma unroll
    for (int c = 0; c < kGroups; ++c) {
      const uint32_t at = sX + st * Smem::kXBytes + 32u * static_cast<uint32_t>(8 * c + g);
      x[c][0] = ld_shared_v4(at);
      x[c][1] = ld_shared_v4(at + 16u);
    }
    __syncwarp();  // every lane has its part of the stage
    if (issued < count) {
      if (issuer) issue(issued);
      ++issued;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t b[kGroups][2];
#pragma unroll
      for (int c = 0; c < kGroups; ++c) {
        b[c][0] = q8_less_1152((__byte_perm(x[c][q].x, x[c][q].y, sel_x) & 0x00ff00ffu) ^ 0x64806480u);
        b[c][1] = q8_less_1152((__byte_perm(x[c][q].z, x[c][q].w, sel_x) & 0x00ff00ffu) ^ 0x64806480u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // bytes 2j, 2j + 1 of the rows' 16: word j / 2, half j & 1
        const auto word = [&](const uint4& v) {
          return j / 2 == 0 ? v.x : j / 2 == 1 ? v.y : j / 2 == 2 ? v.z : v.w;
        };
        const uint32_t sel = (j & 1) ? 0x7362 : 0x5140;  // [r0.b, r1.b, r0.b+1, r1.b+1]
        const uint32_t lo = __byte_perm(word(w[4 * q]), word(w[4 * q + 1]), sel) ^ 0x80808080u;
        const uint32_t hi = __byte_perm(word(w[4 * q + 2]), word(w[4 * q + 3]), sel) ^ 0x80808080u;
        const uint32_t a0 = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4140));
        const uint32_t a1 = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4342));
        const uint32_t a2 = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4140));
        const uint32_t a3 = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4342));
#pragma unroll
        for (int c = 0; c < kGroups; ++c) mma_f16_16816(acc[j][c], a0, a1, a2, a3, b[c][0], b[c][1]);
      }
    }
  }
  if (done < count && lane == 0) {
    // a wait ran out: let the copies in flight land before the ring is reused or left
    for (int i = done; i < issued; ++i) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar + 8u * (i % kStagesS), static_cast<uint32_t>(i / kStagesS) & 1u) &&
             globaltimer_ns() - t0 < timeout_ns) {
      }
    }
  }
  __syncthreads();  // no copy is in flight any more: the ring becomes the sums' place
  float4* part = reinterpret_cast<float4*>(smem);

  // The warps' sums meet, then the blocks': slot 0 receives the block's sums.
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int c = 0; c < kGroups; ++c)
      part[((warp * 8 + j) * kGroups + c) * 32 + lane] =
          make_float4(acc[j][c][0], acc[j][c][1], acc[j][c][2], acc[j][c][3]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int u = i * 32 * kSmallWarps + static_cast<int>(threadIdx.x);
    float4 v[kSmallWarps];
#pragma unroll
    for (int wv = 0; wv < kSmallWarps; ++wv) v[wv] = part[wv * 8 * kGroups * 32 + u];
#pragma unroll
    for (int wv = 1; wv < kSmallWarps; ++wv) {
      v[0].x += v[wv].x;
      v[0].y += v[wv].y;
      v[0].z += v[wv].z;
      v[0].w += v[wv].w;
    }
    part[u] = v[0];
  }
  if (split > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // a unit is (token group, pair of tiles) of one lane
  constexpr int kUnits = 4 * kGroups * 32;
  for (int u = static_cast<int>(threadIdx.x) * split + rank; u < kUnits;
       u += 32 * kSmallWarps * split) {
    const int ul = u & 31, pr = (u >> 5) & 3, c = u >> 7;
    float4 v[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const uint32_t at = 16u * (((2 * pr + jj) * kGroups + c) * 32 + ul);
        v[r][jj] = r < split ? ld_cluster_f4(mapa_shared(base, static_cast<uint32_t>(r)) + at)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    float s[2][4] = {};
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        s[jj][0] += v[r][jj].x;
        s[jj][1] += v[r][jj].y;
        s[jj][2] += v[r][jj].z;
        s[jj][3] += v[r][jj].w;
      }
    // s[jj] = {row g: tokens 2t, 2t + 1; row g + 8: the same} of tile 2 pr + jj
    const int ug = ul >> 2;
    const int n = n0 + 16 * ((ug >> 1) | ((ug & 1) << 2)) + 4 * pr;
    if (n >= p.N) continue;
    const float4 ws = __ldg(reinterpret_cast<const float4*>(p.w_s + n));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int m = 8 * c + 2 * (ul & 3) + e;
      if (m >= p.M) continue;
      const float as = __ldg(p.a_s + m);
      const size_t off = static_cast<size_t>(m) * p.N + n;
      const uint2 zr = p.z != nullptr ? __ldg(reinterpret_cast<const uint2*>(p.z + off))
                                      : make_uint2(0u, 0u);
      const uint2 o =
          make_uint2(pack_bf16x2(fmaf(as * s[0][e], ws.x, bf16lo(zr.x)),
                                 fmaf(as * s[0][2 + e], ws.y, bf16hi(zr.x))),
                     pack_bf16x2(fmaf(as * s[1][e], ws.z, bf16lo(zr.y)),
                                 fmaf(as * s[1][2 + e], ws.w, bf16hi(zr.y))));
      *reinterpret_cast<uint2*>(p.y + off) = o;
    }
  }
  if (split > 1) cluster_sync_all();  // no block leaves while another reads its shared memory
}

}  // namespace coda
