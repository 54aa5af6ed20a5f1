// q8_mid.cuh -- the INT8 product for tens to about two thousand tokens: W widened on its way
// to the tensor cores.
//
//   y[m, n] = a_s[m] w_s[n] sum_k a[m, k] W[k, n] (+ z),   W [K, N] INT8
//
// tcgen05 has no INT8 form on sm_103a, so W has to reach it in 16 bits.  Widening it in
// memory first costs 3 bytes of HBM traffic per code before the product reads it again, which for
// few tokens is most of the time (M = 64, K = 4096, N = 14336: 66 us against a floor of 9).
// Here W stays INT8 as far as shared memory and is widened between there and tensor
// memory, from where tcgen05.mma takes its first operand:
//   D[channel, token] = W^T[channel, k] (tensor memory) * a^T[k, token] (shared memory)
// so a CTA pair (tcgen05 .cta_group::2) owns 256 channels, 128 lanes of tensor memory in each
// CTA, and up to 384 tokens, half of which each CTA holds for both.  Shared memory then sees a
// code of W twice (TMA in, read out) and not the 16-bit form at all: with the operand in shared
// memory instead it would be written and read there too, three times the traffic.  256 tokens
// take 64 KB of it per step of 64 rows (W 16, the tokens' codes 16, widened 32), as long at 128
// bytes a cycle as their products, 512 cycles.  Single CTAs, each with all the tokens, would
// move 112 KB.
//
// The tokens' codes are widened by other warps from shared memory to shared memory, in every
// block that uses them.  A pass of their own before the product spared shared memory that work,
// but was a second launch and a workspace, 5 us of host time: 38 x 112 x 4960 as called 28 us
// with it and 20 without, captured 64 x 4096 x 14336 20.2 us and 19.0, 333 tokens of it 36.3 and
// 35.0, 1024 tokens 84.7 and 88.5, 128 x 4096 x 28672 33.4 and 37.3 (the way out as it was then).
//
// One block of 576 threads per SM, or two of 448 where a pair has at most 128 tokens and there is
// more than one wave of them (kNarrow: half the tensor memory and shared memory); in each CTA:
//   warp 0      TMA producer: a ring of stages of W (128 channels x 64 rows, 8 KB) and of this
//               CTA's half of the tokens (x 64 codes), INT8
//   warp 1      allocates tensor memory; in CTA 0 one thread issues tcgen05.mma (M = 256, N =
//               tokens, K = 16; two of them above 256 tokens) from slots: 32 columns of tensor
//               memory (W) and a swizzled tile of shared memory (the tokens)
//   warps 2..9  widen their quadrant's 32 channels of a stage of W into a slot, two sets of
//               four warps taking the stages in turn; after the last stage they are the epilogue
//   warps 10..  widen a stage's tokens into a slot, two sets in turn of as many warps as have
//               four chunks of 16 codes per lane (64 tokens each, at most four; two in kNarrow):
//               with 256 tokens four took 28.6 us and two 31.5, with 128 two 23.2 and one 27.6,
//               with 64 one 18.9 and two 19.1 (K = 4096, N = 14336)
// Stages and slots are even in number, so that each always belongs to the same sets: a set that
// met one in the next round while the other set still owed it the round before could not
// tell the two by the parity of its barrier.
// All warps of both CTAs that fill a slot arrive on CTA 0's `ready` barrier of it and one
// commit frees it in both CTAs.  The issuing thread is what few tokens wait for: a step takes it
// about 400 cycles (64 tokens' products take 128; W's 8 KB are 350 cycles of an SM's share of
// HBM).  It was 630 with one lane in a branch of its own, where descriptors are not
// warp-uniform.
//
// Widening: a code becomes fp16 by its bits, 0x6400 | (code + 128) = 1024 + 128 + code, and a
// packed subtraction of 1152 leaves it exactly.  A thread (g = lane / 4, t = lane % 4) reads
// the four channels 4 g + b of rows 4 t .. 4 t + 3 of each 16, so that its words are its own
// operands in the store's 16-lane x 256-bit form: channel 4 g + b goes to lane g + 8 b.
// For t >= 2 the rows are read as 2, 3, 0, 1, which with the 128-byte swizzle gives every
// read 32 banks; the k order that follows (k 8..15 of each 16 as 10 11 8 9 14 15 12 13) is
// the same in the tokens' fp16 form, and a sum does not mind.  A lane widens 16 codes of a token
// at a time (16 bytes in, two swizzled 16-byte groups out), free of bank conflicts both ways.
//
// Small N leaves SMs idle, so a cluster of up to four pairs may share a tile along K.  The
// fp32 sums go to shared memory as [token][channel] and each CTA adds and writes its share of
// the tokens, whole rows of its 128 channels, in a fixed order.
#pragma once

#include "q8_small.cuh"

namespace coda {

constexpr int kMidChannels = 128;
constexpr int kMidK = 64;  // rows of W per stage
constexpr uint32_t kMidWBytes = kMidK * kMidChannels;  // 8 KB

__host__ __device__ constexpr int mid_threads(bool narrow) { return narrow ? 448 : 576; }
constexpr int kMidMaxTokens = 384;     // per CTA pair
constexpr int kMidMaxStages = 12;      // of the ring of codes (per CTA)
constexpr int kMidMaxSplit = 4;        // CTA pairs per tile along K
constexpr int kMidMaxSlots = 8;        // of widened codes

// kNarrow: at most 128 tokens per pair and room for two blocks on an SM.
template <bool kNarrow>
struct MidShape {
  static constexpr int kTokens = kNarrow ? 128 : kMidMaxTokens;
  static constexpr uint32_t kCols = kNarrow ? 256 : 512;         // tensor memory: the sums, the slots
  static constexpr uint32_t kRings = kNarrow ? 110592 : 221184;  // shared memory of both rings
  static constexpr uint32_t kBytes = kRings + 512 + 1024;        // barriers, 1 KB alignment slack
  static_assert(kTokens % 32 == 0 && kTokens + 32 * 4 <= static_cast<int>(kCols), "tensor memory");
  static_assert(kTokens * kMidChannels * 4 <= kRings, "the sums overflow the rings");
  static_assert(kBytes <= (kNarrow ? 115712u : 232448u), "blocks per SM");
};
static_assert(8 * (2 * kMidMaxStages + 2 * kMidMaxSlots + 1) + 8 <= 512, "barrier area");

struct MidQ8Params {
  const float* a_s;        // [M]
  const float* w_s;        // [N]
  const __nv_bfloat16* z;  // [M, N] or null
  __nv_bfloat16* y;        // [M, N]
  int M, K, N;
  int tokens;  // per CTA pair: a multiple of 16, of 32 above 256
  int parts;   // instructions of tokens / parts tokens per 16 rows of K: 2 above 256, else 1
  int split;   // CTA pairs per tile along K (the cluster)
  int pairs_stages;  // pairs of stages of codes, at most kMidMaxStages / 2
  int tok_warps;     // warps that widen a stage's tokens
  int pairs_slots;   // pairs of slots, at most kMidMaxSlots / 2
};

// Bytes of a stage of codes (W's, then the half of the tokens; whole swizzle atoms) and of a slot's
// tile of tokens.
__host__ __device__ constexpr uint32_t mid_stage_bytes(int tokens) {
  return kMidWBytes + (static_cast<uint32_t>(tokens / 2 * kMidK) + 1023u) / 1024u * 1024u;
}
__host__ __device__ constexpr uint32_t mid_slot_bytes(int tokens) {
  return static_cast<uint32_t>(tokens / 2 * kMidK * 2);
}

// 16 lanes x 32 columns of tensor memory: thread (g, t) writes columns 8 i + 2 t, 8 i + 2 t + 1
// of lane g from v[4 i], v[4 i + 1] and of lane g + 8 from v[4 i + 2], v[4 i + 3].
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// D[tmem of both CTAs] (+)= A[tmem of both CTAs] * B[smem of both CTAs], fp16 operands; M = 256
// split by rows across the pair, B by its N rows; issued by one thread of CTA 0.
__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor for kind::f16 with fp16 A and B (format code 0), both K-major, and an
// fp32 accumulator; same field positions as idesc_bf16_f32.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// Arrive on a barrier of either CTA without ordering this thread's memory accesses: for handing over
// tensor memory alone, whose writes tcgen05.wait::st has completed and whose order with the other
// CTA's products the tcgen05 fences keep.  A release at cluster scope here took 1450 cycles.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// Arrive on a barrier of either CTA; what this CTA's threads wrote to their own shared memory and
// fenced for the async proxy is the tensor cores' to read.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Generic writes of this thread to shared memory become visible to the async proxy.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A position in a ring of n stages (or slots) and the parity of the round it is in.
struct RingPos {
  int s, n;
  uint32_t ph = 0;
  __device__ __forceinline__ RingPos(int start, int n_) : s(start), n(n_) {
    if (s >= n) s -= n, ph = 1u;
  }
  __device__ __forceinline__ void step(int by) {  // by <= n
    s += by;
    if (s >= n) s -= n, ph ^= 1u;
  }
};

template <bool kNarrow>
__global__ void __launch_bounds__(mid_threads(kNarrow), kNarrow ? 2 : 1)
    product_q8_mid_kernel(const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmX, const MidQ8Params p,
                          uint64_t timeout_ns) {
  constexpr int kMidThreads = mid_threads(kNarrow);
  constexpr uint32_t kMidRings = MidShape<kNarrow>::kRings, kMidCols = MidShape<kNarrow>::kCols;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  // barriers: stage full | stage empty | slot ready | slot free | done, then the TMEM address
  // holder and the abort flag
  const uint32_t bar_full = base + kMidRings;
  const uint32_t bar_empty = bar_full + 8u * kMidMaxStages;
  const uint32_t bar_ready = bar_empty + 8u * kMidMaxStages;
  const uint32_t bar_free = bar_ready + 8u * kMidMaxSlots;
  const uint32_t bar_done = bar_free + 8u * kMidMaxSlots;
  constexpr uint32_t kAfterBars = kMidRings + 8 * (2 * kMidMaxStages + 2 * kMidMaxSlots + 1);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kAfterBars);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + kAfterBars + 4);
  const WaitCtl wc{timeout_ns, &g_coda_status, abort_flag};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0u;
    for (int s = 0; s < kMidMaxStages; ++s) {
      mbar_init(bar_full + 8u * s, 1);
      mbar_init(bar_empty + 8u * s, 4 + p.tok_warps);  // the warps that read the stage
    }
    for (int s = 0; s < kMidMaxSlots; ++s) {
      mbar_init(bar_ready + 8u * s, 2 * (4 + p.tok_warps));  // the same warps, of both CTAs
      mbar_init(bar_free + 8u * s, 1);
    }
    mbar_init(bar_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), kMidCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // barriers of every CTA initialised, tensor memory allocated in all
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const uint32_t tmem_slots = tmem_base + static_cast<uint32_t>((p.tokens + 31) / 32 * 32);
  griddep_launch_dependents();

  // this pair's tile: the token tiles of one channel tile are neighbours in the grid
  // (the cluster rank by the block's index: a value that is known to be the same in all threads)
  const uint32_t cr = blockIdx.x % static_cast<uint32_t>(2 * p.split);
  const uint32_t half = cr & 1u;        // this CTA of the pair: its channels, its half of the tokens
  const uint32_t lead = cr & ~1u;       // cluster rank of the pair's CTA 0
  const int rank = static_cast<int>(cr >> 1);  // part of K
  const int tile = static_cast<int>(blockIdx.x) / (2 * p.split);
  const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);
  const int mt = (p.M + p.tokens - 1) / p.tokens;
  const int n0 = tile / mt * (2 * kMidChannels) + static_cast<int>(half) * kMidChannels;
  const int m0 = tile % mt * p.tokens;
  // its stages of K: kb0 .. kb0 + nkb - 1
  const int stages = 2 * p.pairs_stages, slots = 2 * p.pairs_slots;
  const int nk = (p.K + kMidK - 1) / kMidK;
  const int kb0 = static_cast<int>(static_cast<long long>(nk) * rank / p.split);
  int nkb = static_cast<int>(static_cast<long long>(nk) * (rank + 1) / p.split) - kb0;
  bool paired = true;
  if constexpr (kNarrow) {
    // One address serves both CTAs of the pair.  The two allocate together and get the same columns:
    // 0.9 million pairs did, among other pairs and beside blocks of one CTA that held columns of one of
    // the two SMs alone (columns 0..255 there: both got 256).  PTX does not state it, so it is
    // looked at: otherwise the failure is recorded, nothing is multiplied and the sums are NaN.
    paired = ld_cluster_u32(mapa_shared(smem_u32(tmem_holder), cr ^ 1u)) == tmem_base;
    if (!paired) {
      record_failure(wc, kSitePairTmem);
      nkb = 0;
    }
  }

  const int n_mma = p.tokens / p.parts;  // tokens of one instruction
  const uint32_t stage_bytes = mid_stage_bytes(p.tokens), slot_bytes = mid_slot_bytes(p.tokens);
  const uint32_t sX = base + static_cast<uint32_t>(stages) * stage_bytes;  // the slots' tokens
  const bool issuer = elect_one();
  // While the kernel before this one finishes, the ring's first boxes of W are brought into L2
  // (the point of coherence: nothing is read into this kernel yet).
  if (warp == 0 && issuer)
    for (int i = 0; i < min(nkb, stages); ++i) tma_prefetch_l2_2d(&tmW, n0, (kb0 + i) * kMidK);
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int box = n_mma / 2, row = m0 + static_cast<int>(half) * box;
    const uint32_t bytes = kMidWBytes + static_cast<uint32_t>(p.tokens / 2 * kMidK);
    RingPos r(0, stages);
    int i = 0;
    for (; i < nkb; ++i, r.step(1)) {
      if (!__all_sync(0xffffffffu,
                      bounded_wait(bar_empty + 8u * r.s, r.ph ^ 1u, wc, kSiteProducerEmpty)))
        break;
      const int k = (kb0 + i) * kMidK;
      if (!checked(tma_start_ok(n0, k, p.N, p.K, 1), kChkTmaB) ||
          !checked(tma_start_ok(k, m0, p.K, p.M, 1), kChkTmaA)) {
        *wc.abort_flag = 1u;
        break;
      }
      if (issuer) {
        const uint32_t full = bar_full + 8u * r.s, dst = base + r.s * stage_bytes;
        mbar_arrive_expect_tx(full, bytes);
        tma_load_2d(dst, &tmW, full, n0, k);
        // an instruction's tokens: the first half of them in CTA 0, the second in CTA 1
        tma_load_2d(dst + kMidWBytes, &tmX, full, k, row);
        if (p.parts > 1)
          tma_load_2d(dst + kMidWBytes + static_cast<uint32_t>(box * kMidK), &tmX, full, k,
                      row + n_mma);
      }
      __syncwarp();
    }
    land_copies(bar_full, i, stages, timeout_ns);  // also if others gave up
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the steps and one elected thread issues (here and in the producers),
    // so that descriptors and addresses stay warp-uniform.
    if (half == 0) {
      const uint32_t idesc = idesc_f16_f32(2 * kMidChannels, n_mma);
      const uint64_t desc0 = sdesc_sw128(sX, 16, 1024);
      RingPos r(0, slots);
      for (int i = 0; i < nkb; ++i, r.step(1)) {
        if (!__all_sync(0xffffffffu,
                        bounded_wait(bar_ready + 8u * r.s, r.ph, wc, kSiteMmaFull)))
          break;
        tc_fence_after();
        const uint32_t a0 = tmem_slots + 32u * r.s;
        // shared memory ends below 2^18, so the address field (address / 16) takes the sums
        const uint64_t b0 = desc0 + r.s * slot_bytes / 16;
        if (issuer) {
#pragma unroll
          for (int k = 0; k < kMidK / 16; ++k)
            umma_f16_ts_pair(tmem_base, a0 + 8u * k, b0 + 2u * k, idesc, (i | k) != 0 ? 1u : 0u);
          if (p.parts > 1) {
            const uint64_t b1 = b0 + static_cast<uint32_t>(n_mma / 2) * kMidK * 2 / 16;
#pragma unroll
            for (int k = 0; k < kMidK / 16; ++k)
              umma_f16_ts_pair(tmem_base + n_mma, a0 + 8u * k, b1 + 2u * k, idesc,
                               (i | k) != 0 ? 1u : 0u);
          }
          umma_commit_pair_mc(bar_free + 8u * r.s, pair_mask);
        }
        __syncwarp();
      }
      // every product issued here (also after a wait that ran out)
      if (issuer) umma_commit_pair_mc(bar_done, pair_mask);
    }
    __syncwarp();
  } else if (warp >= 10 + 2 * p.tok_warps) {
    // nothing to widen
  } else if (warp >= 10) {
    // ------------------------------------------------------------ widening the tokens
    const int set = (warp - 10) & 1, first = (warp - 10) / 2 * 32 + lane;
    const int chunks = p.tokens / 2 * 4;  // 16 codes each, four to a row
    const uint32_t ready0 = mapa_shared(bar_ready, lead);
    RingPos r(set, stages), slot(set, slots);
    for (int i = set; i < nkb; i += 2, r.step(2), slot.step(2)) {
      if (!__all_sync(0xffffffffu,
                      bounded_wait(bar_full + 8u * r.s, r.ph, wc, kSiteEpiTmemFull) &&
                          bounded_wait(bar_free + 8u * slot.s, slot.ph ^ 1u, wc, kSiteMmaTmemEmpty)))
        break;
      const uint32_t src = base + r.s * stage_bytes + kMidWBytes, dst = sX + slot.s * slot_bytes;
      for (int q0 = first; q0 < chunks; q0 += 4 * 32 * p.tok_warps) {  // four reads under way
        uint4 v[4];
#pragma unroll
        for (int b = 0; b < 4; ++b)
          v[b] = ld_shared_v4(
              src + 16u * static_cast<uint32_t>(min(q0 + 32 * p.tok_warps * b, chunks - 1)));
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t q = static_cast<uint32_t>(q0 + 32 * p.tok_warps * b);
          if (q >= static_cast<uint32_t>(chunks)) break;
          const uint32_t row = q >> 2, c = q & 3u;
          const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
          uint32_t o[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t u = w[k] ^ 0x80808080u;
            o[2 * k] = q8_less_1152(__byte_perm(u, 0x64646464u, 0x4140));
            o[2 * k + 1] = q8_less_1152(__byte_perm(u, 0x64646464u, 0x4342));
          }
          const uint32_t line = dst + 128u * row;
          st_shared_v4(line + 16u * ((2u * c) ^ (row & 7u)), o[0], o[1], o[2], o[3]);
          st_shared_v4(line + 16u * ((2u * c + 1u) ^ (row & 7u)), o[5], o[4], o[7], o[6]);
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_empty + 8u * r.s);
        mbar_arrive_remote(ready0 + 8u * slot.s);
      }
    }
  } else {
    // ------------------------------------------------------------ widening W
    const uint32_t quad = warp & 3;
    const uint32_t g = lane >> 2, t = lane & 3;
    // this thread's word of row r of 16: chunk (2 quad + g / 4) ^ (r % 8), word g % 4
    const uint32_t chunk = 2 * quad + (g >> 2);
    uint32_t at[4];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
      const uint32_t r = 4 * t + (t >= 2 ? j ^ 2u : j);
      at[j] = 128u * r + 16u * (chunk ^ (r & 7u)) + 4u * (g & 3u);
    }
    const int set = (warp - 2) >> 2;  // set 0: even stages, set 1: odd ones
    RingPos r(set, stages), slot(set, slots);
    for (int i = set; i < nkb; i += 2, r.step(2), slot.step(2)) {
      if (!__all_sync(0xffffffffu,
                      bounded_wait(bar_full + 8u * r.s, r.ph, wc, kSiteEpiTmemFull)))
        break;
      const uint32_t src = base + r.s * stage_bytes;
      uint32_t l[4][4];
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) l[c][j] = ld_shared_u32(src + 2048u * c + at[j]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty + 8u * r.s);
      uint32_t v01[16], v23[16];  // channels 0, 1 (lanes g, g + 8) and 2, 3 (g + 16, g + 24)
#pragma unroll
      for (uint32_t c = 0; c < 4; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // columns 8 c + 2 t + h
          const uint32_t lo = __byte_perm(l[c][2 * h], l[c][2 * h + 1], 0x5140) ^ 0x80808080u;
          const uint32_t hi = __byte_perm(l[c][2 * h], l[c][2 * h + 1], 0x7362) ^ 0x80808080u;
          v01[4 * c + h] = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4140));
          v01[4 * c + 2 + h] = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4342));
          v23[4 * c + h] = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4140));
          v23[4 * c + 2 + h] = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4342));
        }
      // the slot's earlier products are done
      if (!__all_sync(0xffffffffu,
                      bounded_wait(bar_free + 8u * slot.s, slot.ph ^ 1u, wc, kSiteMmaTmemEmpty)))
        break;
      tc_fence_after();
      const uint32_t dst = tmem_slots + 32u * slot.s + (quad * 32u << 16);
      tmem_st_16x256b_x4(dst, v01);
      tmem_st_16x256b_x4(dst + (16u << 16), v23);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(bar_ready + 8u * slot.s, lead));
    }
  }

  // ------------------------------------------------------------ epilogue
  // The sums leave tensor memory as [token][channel] in the ring's place.
  if (warp >= 2 && warp < 10) {
    const bool ok = bounded_wait(bar_done, 0, wc, kSiteDrain);
    if (__all_sync(0xffffffffu, ok) && paired) {
      tc_fence_after();
      const uint32_t quad = warp & 3;
      const uint32_t ch = 32 * quad + 4 * (lane & 7) + (lane >> 3);  // the channel in this lane
      for (int c = 32 * ((warp - 2) >> 2); c < p.tokens; c += 64) {  // two warps share a quadrant
        uint32_t v[32];
        tmem_ld32(tmem_base + (quad * 32u << 16) + static_cast<uint32_t>(c), v);
        tmem_ld_wait(v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c + j < p.tokens) st_shared_u32(base + 4u * ((c + j) * kMidChannels + ch), v[j]);
      }
      tc_fence_before();
    } else if (!paired) {
      for (int i = static_cast<int>(threadIdx.x) - 64; i < p.tokens * kMidChannels; i += 256)
        st_shared_u32(base + 4u * static_cast<uint32_t>(i), 0x7fffffffu);  // NaN
    }
  } else if (warp == 1) {
    // both CTAs: no TMEM release while products may still write it
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(bar_done, 0)) {
        if (globaltimer_ns() - t0 > timeout_ns) {
          record_failure(wc, kSiteDrain);
          break;
        }
      }
    }
    __syncwarp();
  }
  // A thread keeps its 8 channels and takes every (threads / 16)-th of this block's tokens, which
  // are rank, rank + split, ...  What it reads for two tokens is under way together (1024 x
  // 4096 x 14336, three waves: 82.5 us, one token at a time 87; four at a time no faster).
  static_assert(kMidThreads % (kMidChannels / 8) == 0, "a thread keeps its channels");
  constexpr int kU = 2, kStride = kMidThreads / (kMidChannels / 8);
  const int c8 = static_cast<int>(threadIdx.x) % (kMidChannels / 8) * 8, n = n0 + c8;
  float ws[8] = {};
  if (n < p.N) {
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(p.w_s + n));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(p.w_s + n + 4));
    ws[0] = w0.x, ws[1] = w0.y, ws[2] = w0.z, ws[3] = w0.w;
    ws[4] = w1.x, ws[5] = w1.y, ws[6] = w1.z, ws[7] = w1.w;
  }
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kMidCols);

  const int tokens = min(p.tokens, p.M - m0);
  const int mine = n < p.N && tokens > rank ? (tokens - rank + p.split - 1) / p.split : 0;
  // the eight lanes that read shared memory together take different halves of their 32 bytes
  const uint32_t hi = (lane >> 2) & 1;
  for (int i0 = static_cast<int>(threadIdx.x) / (kMidChannels / 8); i0 < mine; i0 += kU * kStride) {
    float as[kU], v[kU][8] = {};
    Chunk8 z[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool in = i0 + u * kStride < mine;
      const int m = m0 + rank + (i0 + u * kStride) * p.split;
      as[u] = in ? __ldg(p.a_s + m) : 0.f;
      if (in && p.z != nullptr) z[u] = ldg8(p.z + static_cast<size_t>(m) * p.N + n);
    }
#pragma unroll 1
    for (int r = 0; r < p.split; ++r) {
      const uint32_t peer = mapa_shared(base, 2u * static_cast<uint32_t>(r) + half);
      float4 a[kU], b[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int tok = rank + (i0 + u * kStride) * p.split;
        const uint32_t at = peer + 4u * static_cast<uint32_t>(tok * kMidChannels + c8);
        a[u] = b[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + u * kStride < mine) {
          a[u] = ld_cluster_f4(at + 16u * hi);
          b[u] = ld_cluster_f4(at + 16u - 16u * hi);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const float4 lo4 = hi ? b[u] : a[u], hi4 = hi ? a[u] : b[u];
        v[u][0] += lo4.x, v[u][1] += lo4.y, v[u][2] += lo4.z, v[u][3] += lo4.w;
        v[u][4] += hi4.x, v[u][5] += hi4.y, v[u][6] += hi4.z, v[u][7] += hi4.w;
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (i0 + u * kStride >= mine) break;
      const int m = m0 + rank + (i0 + u * kStride) * p.split;
      float zv[8] = {};
      if (p.z != nullptr) unpack8(z[u], zv);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_bf16x2(fmaf(as[u] * v[u][2 * e], ws[2 * e], zv[2 * e]),
                           fmaf(as[u] * v[u][2 * e + 1], ws[2 * e + 1], zv[2 * e + 1]));
      stg8(p.y + static_cast<size_t>(m) * p.N + n, o);
    }
  }
  cluster_sync_all();  // no block leaves while another reads its shared memory or its barriers
}

}  // namespace coda
