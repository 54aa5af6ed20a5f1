// attn_q8_tile.cuh -- attention over the 8-bit paged cache for many rows (chunks and whole prompts): tiles of
// 256 packed rows on tcgen05.
//
// A block holds two tiles of 128 rows of q (fp16, shared memory) and walks the keys 128 at a time:
//   S_w = q_w k^T     128 x 128, tensor memory, fp32     (w = 0, 1: the two tiles)
//   P_w = 2^(S_w scale - base) * v's scale, fp16, over the first half of S_w
//   o_w += P_w v      128 x D, tensor memory; P_w is the first operand, from tensor memory
// The tensor cores see codes widened to fp16 (exact); k's scales multiply S's columns and v's P's, in the
// softmax.  Bound by the tensor cores: 4 * 256 * 128 * D operations per unit, 2048 cycles for D = 128; its 32768
// exponentials are half of that, and the widening of 32768 codes, once per 256 rows, a fifth of the issue slots.
//
// One block of 384 threads per SM (three warps to a quarter of it: 168 registers each):
//   warps 0..3, 4..7   softmax of tile 0, 1: a warp has 32 rows (its quarter of tensor memory's lanes), a thread 32
//                      columns of four of them.  S is read twice, for the maximum and for the exponentials.
//   warps 8..10        widen k and v from global memory into shared memory, rings of two tiles each, in groups of 16
//                      keys dealt in turn; a group's codes are loaded to registers a unit ahead
//   warp 11            issues tcgen05.mma:  S_0(j + 1) behind P_0(j) v, S_1(j + 1) behind P_1(j) v, so that one tile's
//                      softmax runs beside the other's products
// o is rescaled only where a row's maximum has grown by more than 2^8 (P stays below fp16's largest): hardly ever
// after the first units.
#pragma once

#include "attn_q8.cuh"
#include "q8_mid.cuh"

namespace coda {

constexpr int kTileRows = 256, kTileThreads = 384;
constexpr int kTileStages = 2, kTileScales = 4;  // rings: of k's and v's tiles, of their scales
constexpr uint32_t kSiteAttn = 12;               // of bounded waits: kSiteAttn + which

template <int kD>
struct TileSmem {
  static constexpr uint32_t kOperand = 128 * kD * 2;  // 128 rows of fp16: panels of 64 columns
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kOperand;
  static constexpr uint32_t kV = kK + kTileStages * kOperand;
  static constexpr uint32_t kScale = kV + kTileStages * kOperand;  // [slot][k's 128, v's 128, the largest of v's]
  static constexpr uint32_t kScaleSlot = 2 * 512 + 16;
  static constexpr uint32_t kBar = kScale + kTileScales * kScaleSlot;
  static constexpr uint32_t kBars = 4 * kTileStages + 2 * kTileScales + 8 + 1;
  static constexpr uint32_t kRow = kBar + 8 * kBars + 8;  // a number or two per row, from thread to thread
  static constexpr uint32_t kEnd = kRow + 256 * 8;  // tensor memory's address, the abort flag
  static constexpr uint32_t kUsed = kEnd + 16;
  // (the sequences' units at the start take the place of q, k and v)
  static constexpr uint32_t kBytes = (kUsed > 65536 ? kUsed : 65536) + 1024;
  static_assert(kBytes <= 232448u - 1024u, "shared memory");
};

// D[tmem] (+)= A[tmem] * B[smem], fp16
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 lanes x 32 columns of tensor memory: thread (g, t) reads columns 8 i + 2 t, 8 i + 2 t + 1 of lane g into
// v[4 i], v[4 i + 1] and of lane g + 8 into v[4 i + 2], v[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// 16 lanes x 16 columns: thread (g, t) writes column 4 i + t of lane g from v[2 i] and of lane g + 8 from v[2 i + 1].
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait16(uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                 "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]), "+r"(a[15]),
                 "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                 "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]), "+r"(b[15])
               :
               : "memory");
}

// A warp's 32 lanes x 32 columns: rows g + 8 k in v[k / 2][4 i + 2 (k % 2) + e], columns 8 i + 2 t + e.
struct Block32 {
  uint32_t v[2][16];
  __device__ __forceinline__ void load(uint32_t taddr) {
    tmem_ld_16x256b_x4(taddr, v[0]);
    tmem_ld_16x256b_x4(taddr + (16u << 16), v[1]);
  }
  __device__ __forceinline__ void wait() { tmem_ld_wait16(v[0], v[1]); }
  __device__ __forceinline__ uint64_t pair(int i, int k) const {
    return pack2(__uint_as_float(v[k / 2][4 * i + 2 * (k % 2)]), __uint_as_float(v[k / 2][4 * i + 2 * (k % 2) + 1]));
  }
};

// What other threads wrote to shared memory before a barrier is seen by the tensor cores.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Where the 16-byte group c (8 values) of a row sits in an operand of panels of 64 columns, 128-byte
// swizzle: the layout of both the K-major operands (q, k) and the one whose rows are k (v).
__device__ __forceinline__ uint32_t panel_at(uint32_t row, uint32_t c) {
  return (c >> 3) * 16384u + row * 128u + (((c & 7u) ^ (row & 7u)) << 4);
}

// The softmax's two walks over a warp's 32 rows of S, 32 columns at a time with the next 32 on their way; `a` holds
// the first 32 between them.  A thread has 8 columns of four rows, so a column's scale, read once, serves four
// products: with a row to a thread, the reads of scales alone took as long on shared memory as the operands of
// the products.  `ts`: the warp's place in tensor memory.  `sc`: k's 128 scales (v's 128 numbers on) from
// column 2 t.  kEdge: row k sees columns 0 .. seen[k] of those from 2 t on.
template <bool kEdge>
__device__ __forceinline__ void largest_of_32(const Block32& s, const float* sc, const int (&seen)[4], int c,
                                              float (&mx)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 k2 = *reinterpret_cast<const float2*>(sc + c + 8 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x, y;
      unpack2(mul2(s.pair(i, k), pack2(k2.x, k2.y)), x, y);
      if constexpr (kEdge) {
        if (c + 8 * i > seen[k]) x = -INFINITY;
        if (c + 8 * i + 1 > seen[k]) y = -INFINITY;
      }
      mx[k] = max3(mx[k], x, y);
    }
  }
}

template <bool kEdge>
__device__ __forceinline__ void largest_scores(uint32_t ts, const float* sc, const int (&seen)[4], Block32& a, Block32& b,
                                               float (&mx)[4]) {
  a.load(ts);
  a.wait();
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    b.load(ts + c + 32);
    largest_of_32<kEdge>(a, sc, seen, c, mx);
    b.wait();
    a.load(ts + (c + 64) % 128);
    largest_of_32<kEdge>(b, sc, seen, c + 32, mx);
    a.wait();
  }
}

// P = 2^(S k's scale rf - less) v's scale, in fp16 over columns of S that have been read; the sums without v's.
template <bool kEdge>
__device__ __forceinline__ void weights_of_32(const Block32& s, uint32_t ts, const float* sc, const int (&seen)[4], int c,
                                              const float (&rf)[4], const float (&less)[4], uint64_t (&sum)[4]) {
  uint32_t pk[2][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 k2 = *reinterpret_cast<const float2*>(sc + c + 8 * i);
    const float2 v2 = *reinterpret_cast<const float2*>(sc + 128 + c + 8 * i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x, y;
      unpack2(fma2(mul2(s.pair(i, k), pack2(k2.x, k2.y)), pack2(rf[k], rf[k]), pack2(-less[k], -less[k])), x, y);
      x = ex2(x);
      y = ex2(y);
      if constexpr (kEdge) {
        if (c + 8 * i > seen[k]) x = 0.f;
        if (c + 8 * i + 1 > seen[k]) y = 0.f;
      }
      const uint64_t xy = pack2(x, y);
      sum[k] = add2(sum[k], xy);
      unpack2(mul2(xy, pack2(v2.x, v2.y)), x, y);
      if constexpr (kEdge) {  // (a scale behind the row's last key may be NaN)
        if (c + 8 * i > seen[k]) x = 0.f;
        if (c + 8 * i + 1 > seen[k]) y = 0.f;
      }
      pk[k / 2][2 * i + k % 2] = pack_f16x2(x, y);
    }
  }
  tmem_st_16x128b_x4(ts + c / 2, pk[0]);
  tmem_st_16x128b_x4(ts + c / 2 + (16u << 16), pk[1]);
}

template <bool kEdge>
__device__ __forceinline__ void weights(uint32_t ts, const float* sc, const int (&seen)[4], const float (&rf)[4],
                                        const float (&less)[4], Block32& a, Block32& b, uint64_t (&sum)[4]) {
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    b.load(ts + c + 32);
    weights_of_32<kEdge>(a, ts, sc, seen, c, rf, less, sum);
    b.wait();
    if (c == 0) a.load(ts + 64);
    weights_of_32<kEdge>(b, ts, sc, seen, c + 32, rf, less, sum);
    a.wait();
  }
}

template <int kD>
__global__ void __launch_bounds__(kTileThreads, 1)
    attn_q8_tile_kernel(const AttnQ8Params p, const AttnWs ws, const AttnDeal deal, uint64_t timeout_ns) {
  using Smem = TileSmem<kD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int places = p.batch.width << p.cache.page_log2;
  const uint32_t bars = base + Smem::kBar;
  const auto k_full = [&](uint32_t s) { return bars + 8u * s; };
  const auto k_empty = [&](uint32_t s) { return bars + 8u * (kTileStages + s); };
  const auto v_full = [&](uint32_t s) { return bars + 8u * (2 * kTileStages + s); };
  const auto v_empty = [&](uint32_t s) { return bars + 8u * (3 * kTileStages + s); };
  const auto sc_full = [&](uint32_t s) { return bars + 8u * (4 * kTileStages + s); };
  const auto sc_empty = [&](uint32_t s) { return bars + 8u * (4 * kTileStages + kTileScales + s); };
  constexpr uint32_t kB = 4 * kTileStages + 2 * kTileScales;
  const auto s_full = [&](uint32_t w) { return bars + 8u * (kB + w); };       // S_w is there
  const auto p_full = [&](uint32_t w) { return bars + 8u * (kB + 2 + w); };   // P_w is there
  const auto pv_done = [&](uint32_t w) { return bars + 8u * (kB + 4 + w); };  // o_w has P_w v
  const auto q_full = [&](uint32_t w) { return bars + 8u * (kB + 6 + w); };
  const uint32_t drained = bars + 8u * (kB + 8);
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Smem::kEnd + 4);
  const WaitCtl wc{timeout_ns, &g_coda_status, abort_flag};
  // a whole warp waits, and gives up, together
  const auto warp_wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, wc, site)) != 0;
  };
  griddep_launch_dependents();
  griddep_wait();

  AttnWalk w;
  int64_t u0, u1;
  const int64_t total =
      walk_start<kTileRows, kTileThreads>(w, p, deal, places, reinterpret_cast<int64_t*>(smem), u0, u1);
  if (tid == 0) ws.cut[blockIdx.x].valid = 0;
  if (u0 >= u1) return;
  if (tid == 0) {
    *abort_flag = 0u;
    for (uint32_t s = 0; s < kTileStages; ++s) {
      mbar_init(k_full(s), 3);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 3);
      mbar_init(v_empty(s), 1);
    }
    for (uint32_t s = 0; s < kTileScales; ++s) {
      mbar_init(sc_full(s), 1);
      mbar_init(sc_empty(s), 8);
    }
    for (uint32_t i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
      mbar_init(pv_done(i), 1);
      mbar_init(q_full(i), 4);
    }
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  if (warp == 11) {
    tmem_alloc(base + Smem::kEnd, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Smem::kEnd);
  const uint32_t count = static_cast<uint32_t>(u1 - u0);

  if (warp >= 8 && warp < 11) {
    // ------------------------------------------------------------- widening
    // Groups of 16 keys, 8 of k and 8 of v: this warp's are every third from `kg` and from `vg`.
    constexpr int kPer = kD / 32;  // of a lane and group, 16 codes each
    const int first = warp - 8;
    const int kg = first, vg = (first + 1) % 3;
    uint4 buf[6][kPer];  // three of k, three of v
    float4 ks, vs;       // warp 9: scales of keys 4 lane .. 4 lane + 3
    // pages of the 8 groups of keys of a unit, one per lane 0..7: looked up a unit before its loads
    const auto pages_at = [&](const AttnWalk& a) {
      const int key = a.unit * kAttnUnit + 16 * (lane & 7);
      return key < a.extent ? page_of(p.batch, p.cache, a.b, key) : -1;
    };
    const int mask = (1 << p.cache.page_log2) - 1;
    int pages = -1, pages_next = pages_at(w), key0 = 0, extent = 0, hk = 0;  // of the unit that is loaded
    uint32_t walked = 0;
    const auto next = [&]() {  // takes over the unit that `w` is at, and moves w to the one behind it
      pages = pages_next;
      key0 = w.unit * kAttnUnit;
      extent = w.extent;
      hk = w.hk;
      if (++walked < count) {
        walk_on<kTileRows>(w, p, deal, places);
        pages_next = pages_at(w);
      }
    };
    // The lane's j-th 16 codes of a group: the eight threads that write together have four neighbouring ones of
    // two rows; with the swizzle, 128 bytes without a bank twice.
    const auto row_at = [&](int j) { return static_cast<uint32_t>(lane >> 2) + 8u * (kD == 128 ? j >> 1 : j); };
    const auto col_at = [&](int j) { return static_cast<uint32_t>(lane & 3) + (kD == 128 ? 4u * (j & 1) : 0u); };
    const auto group = [&](int n) { return n < 3 ? kg + 3 * n : vg + 3 * (n - 3); };  // 8 or more: none
    const auto load = [&](int n) {
      const int g = group(n);
      if (g >= 8) return;
      const int page = __shfl_sync(0xffffffffu, pages, g);
      if (page < 0) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) buf[n][j] = make_uint4(0u, 0u, 0u, 0u);
        return;
      }
      const uint8_t* const q =
          (n < 3 ? p.cache.k_q : p.cache.v_q) + cache_entry(p.cache, page, hk, (key0 + 16 * g) & mask) * kD;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        buf[n][j] = *reinterpret_cast<const uint4*>(q + row_at(j) * kD + 16u * col_at(j));
    };
    const auto widen = [&](int n, uint32_t to) {
      const int g = group(n);
      if (g >= 8) return;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t r = 16u * g + row_at(j), c = 2u * col_at(j);
        uint32_t x[8];
        q8_to_f16x2(buf[n][j].x, x[0], x[1]);
        q8_to_f16x2(buf[n][j].y, x[2], x[3]);
        q8_to_f16x2(buf[n][j].z, x[4], x[5]);
        q8_to_f16x2(buf[n][j].w, x[6], x[7]);
        st_shared_v4(to + panel_at(r, c), x[0], x[1], x[2], x[3]);
        st_shared_v4(to + panel_at(r, c + 1u), x[4], x[5], x[6], x[7]);
      }
    };
    const auto load_scales = [&]() {
      const int page = __shfl_sync(0xffffffffu, pages, lane >> 2), key = key0 + 4 * lane;
      const float lost = __int_as_float(0x7fffffff);  // a page that does not exist: NaN
      ks = vs = make_float4(lost, lost, lost, lost);
      if (page >= 0) {
        const size_t e = cache_entry(p.cache, page, hk, key & mask);
        ks = *reinterpret_cast<const float4*>(p.cache.k_s + e);
        vs = *reinterpret_cast<const float4*>(p.cache.v_s + e);
      }
      const auto cut = [&](float4& s) {  // nothing behind the last key is looked at
        if (key >= extent) s.x = 0.f;
        if (key + 1 >= extent) s.y = 0.f;
        if (key + 2 >= extent) s.z = 0.f;
        if (key + 3 >= extent) s.w = 0.f;
      };
      if (key + 3 >= extent) {
        cut(ks);
        cut(vs);
      }
    };
    next();
    if (first == 1) load_scales();
#pragma unroll
    for (int n = 0; n < 6; ++n) load(n);
    for (uint32_t i = 0; i < count; ++i) {
      const uint32_t st = i % kTileStages, ph = i / kTileStages & 1u;
      const bool more = i + 1 < count;
      if (more) next();
      if (first == 1) {
        const uint32_t sl = i % kTileScales;
        if (!warp_wait(sc_empty(sl), (i / kTileScales & 1u) ^ 1u, kSiteAttn)) break;
        float* const sc = reinterpret_cast<float*>(smem + Smem::kScale + sl * Smem::kScaleSlot);
        *reinterpret_cast<float4*>(sc + 4 * lane) = ks;
        *reinterpret_cast<float4*>(sc + 128 + 4 * lane) = vs;
        const auto size = [](float s) { return fabsf(s) <= 3.402823466e38f ? fabsf(s) : 0.f; };
        const float top = fmaxf(fmaxf(size(vs.x), size(vs.y)), fmaxf(size(vs.z), size(vs.w)));
        const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (lane == 0) sc[256] = __uint_as_float(all);
        __syncwarp();
        if (lane == 0) mbar_arrive(sc_full(sl));
        if (more) load_scales();
      }
      if (!warp_wait(k_empty(st), ph ^ 1u, kSiteAttn + 1)) break;
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        widen(n, base + Smem::kK + st * Smem::kOperand);
        if (more) load(n);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(st));
      if (!warp_wait(v_empty(st), ph ^ 1u, kSiteAttn + 2)) break;
#pragma unroll
      for (int n = 3; n < 6; ++n) {
        widen(n, base + Smem::kV + st * Smem::kOperand);
        if (more) load(n);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
    }
  } else if (warp == 11) {
    // ------------------------------------------------------------- products
    const bool issuer = elect_one();
    constexpr uint32_t kIdescS = idesc_f16_f32(128, 128);
    constexpr uint32_t kIdescO = idesc_f16_f32(128, kD) | (1u << 16);  // v: rows are k
    const auto s_mma = [&](uint32_t t, uint32_t st) {
#pragma unroll
      for (uint32_t k = 0; k < kD / 16; ++k) {
        const uint32_t off = (k / 4) * 16384u + (k % 4) * 32u;
        const uint64_t a = sdesc_sw128(base + Smem::kQ + t * Smem::kOperand + off, 16, 1024);
        const uint64_t b = sdesc_sw128(base + Smem::kK + st * Smem::kOperand + off, 16, 1024);
        if (issuer) umma_bf16(tmem + 128u * t, a, b, kIdescS, k > 0);
      }
      if (issuer) umma_commit(s_full(t));
    };
    const auto o_mma = [&](uint32_t t, uint32_t st, bool first) {
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k) {
        const uint64_t b = sdesc_sw128(base + Smem::kV + st * Smem::kOperand + k * 2048u, 16384, 1024);
        if (issuer) umma_f16_ts(tmem + 256u + kD * t, tmem + 128u * t + 8u * k, b, kIdescO, !first || k > 0);
      }
      if (issuer) umma_commit(pv_done(t));
    };
    const auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t site) {
      const bool ok = warp_wait(bar, parity, site);
      tc_fence_after();
      return ok;
    };
    uint32_t i = 0;
    bool ok = true;
    for (uint32_t items = 0; ok && i < count; ++items) {
      const uint32_t end = i + min(static_cast<uint32_t>(w.units - w.unit), count - i);  // of the item here
      uint32_t st = i % kTileStages;
      ok = wait_all(q_full(0), items & 1u, kSiteAttn + 3) && wait_all(q_full(1), items & 1u, kSiteAttn + 3) &&
           wait_all(k_full(st), i / kTileStages & 1u, kSiteAttn + 4);
      if (!ok) break;
      s_mma(0, st);
      s_mma(1, st);
      if (issuer) umma_commit(k_empty(st));
      for (bool first = true; i < end; ++i, first = false) {
        st = i % kTileStages;
        const uint32_t ph = i / kTileStages & 1u, uph = i & 1u;
        const uint32_t nst = (i + 1) % kTileStages, nph = (i + 1) / kTileStages & 1u;
        const bool more = i + 1 < end;
        ok = wait_all(v_full(st), ph, kSiteAttn + 5) && wait_all(p_full(0), uph, kSiteAttn + 6);
        if (!ok) break;
        o_mma(0, st, first);
        if (more) {
          ok = wait_all(k_full(nst), nph, kSiteAttn + 4);
          if (!ok) break;
          s_mma(0, nst);
        }
        ok = wait_all(p_full(1), uph, kSiteAttn + 6);
        if (!ok) break;
        o_mma(1, st, first);
        if (issuer) umma_commit(v_empty(st));
        if (more) {
          s_mma(1, nst);
          if (issuer) umma_commit(k_empty(nst));
        }
      }
      if (ok && i < count) walk_item<kTileRows>(w, p, deal, places);
    }
    // (no product is left in flight when the tensor memory is given back)
    if (issuer) umma_commit(drained);
    bounded_wait(drained, 0, wc, kSiteAttn + 7);
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const uint32_t tl = static_cast<uint32_t>(warp) >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // its quarter of tensor memory's lanes
    const uint32_t ts = tmem + 128u * tl + lanes, to = tmem + 256u + kD * tl + lanes;
    const uint32_t r = static_cast<uint32_t>(tid) & 127u;  // its row of the tile
    const int t2 = 2 * (lane & 3);
    const float* const scales = reinterpret_cast<const float*>(smem + Smem::kScale);
    // the warp's rows: number lane from the thread that has the row alone, and g + 8 k of those that share it
    float2* const rows = reinterpret_cast<float2*>(smem + Smem::kRow) + 32 * warp;
    uint32_t i = 0;
    bool ok = true;
    while (ok && i < count) {
      // an item, or what of it lies in this block's share: its row of q, in fp16
      const uint32_t begin = i, end = i + min(static_cast<uint32_t>(w.units - w.unit), count - i);
      const AttnRow row = attn_row(p, w.s, w.hk, w.tile * kTileRows + static_cast<int>(128 * tl + r));
      const int low = __shfl_sync(0xffffffffu, row.limit, 0);  // the smallest of the warp's rows
      __syncwarp();
      {
        Chunk8 c[kD / 8];
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < kD / 8; ++j) c[j] = ldg8(p.q + row.at * kD + 8 * j);
#pragma unroll
        for (int j = 0; j < kD / 8; ++j) {
          float v[8];
          unpack8(c[j], v);
#pragma unroll
          for (int e = 0; e < 8; e += 2) amax = max3_abs_nan(amax, v[e], v[e + 1]);
        }
        float up, down;
        row_power(amax, up, down);
        rows[lane] = make_float2(p.scale_log2 * down, __int_as_float(row.limit));
#pragma unroll
        for (int j = 0; j < kD / 8; ++j) {
          float v[8];
          unpack8(c[j], v);
          st_shared_v4(base + Smem::kQ + tl * Smem::kOperand + panel_at(r, j), pack_f16x2(v[0] * up, v[1] * up),
                       pack_f16x2(v[2] * up, v[3] * up), pack_f16x2(v[4] * up, v[5] * up),
                       pack_f16x2(v[6] * up, v[7] * up));
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(tl));
      float m[4], bs[4], rf[4], lv = kLeastScale;
      int limit[4];  // from column 2 t on
      uint64_t sum[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 x = rows[(lane >> 2) + 8 * k];
        rf[k] = x.x;
        limit[k] = __float_as_int(x.y) - t2;
        m[k] = bs[k] = -INFINITY;
        sum[k] = 0;
      }
      int key = w.unit * kAttnUnit;
      for (; i < end; ++i, key += kAttnUnit) {
        const uint32_t uph = i & 1u, sl = i % kTileScales;
        ok = warp_wait(sc_full(sl), i / kTileScales & 1u, kSiteAttn + 8) && warp_wait(s_full(tl), uph, kSiteAttn + 9);
        if (!ok) break;
        tc_fence_after();
        const float* const sc = scales + sl * (Smem::kScaleSlot / 4);
        const bool edge = key + kAttnUnit - 1 > low;
        const int seen[4] = {limit[0] - key, limit[1] - key, limit[2] - key, limit[3] - key};
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        Block32 a, b;
        if (edge)
          largest_scores<true>(ts, sc + t2, seen, a, b, mx);
        else
          largest_scores<false>(ts, sc + t2, seen, a, b, mx);
        lv = fmaxf(lv, scale_power(sc[256]));
        // What is taken out of the exponents: moved where P would leave fp16.
        bool move = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
          mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
          m[k] = fmaxf(m[k], mx[k] == -INFINITY ? mx[k] : mx[k] * rf[k]);
          move |= m[k] + lv > bs[k] + 8.0f;
        }
        if (__any_sync(0xffffffffu, move)) {
          float corr[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            corr[k] = 1.0f;
            if (m[k] + lv > bs[k] + 8.0f) {
              corr[k] = ex2(bs[k] - (m[k] + lv));
              bs[k] = m[k] + lv;
            }
            sum[k] = mul2(sum[k], pack2(corr[k], corr[k]));
          }
          if (i > begin) {
            ok = warp_wait(pv_done(tl), uph ^ 1u, kSiteAttn + 10);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              b.load(to + c);
              b.wait();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  b.v[h][e] = __float_as_uint(__uint_as_float(b.v[h][e]) * corr[2 * h + (e >> 1 & 1)]);
                tmem_st_16x256b_x4(to + c + (16u * h << 16), b.v[h]);
              }
            }
            tmem_st_wait();
          }
        }
        float less[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) less[k] = bs[k] == -INFINITY ? 0.f : bs[k];  // (no key seen yet)
        if (edge)
          weights<true>(ts, sc + t2, seen, rf, less, a, b, sum);
        else
          weights<false>(ts, sc + t2, seen, rf, less, a, b, sum);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full(tl));
          mbar_arrive(sc_empty(sl));
        }
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float x, y;
        unpack2(sum[k], x, y);
        x += y;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (t2 == 0) rows[(lane >> 2) + 8 * k] = make_float2(bs[k], x);
      }
      __syncwarp();
      const float bs_row = rows[lane].x, l = rows[lane].y;
      if (!ok) break;
      ok = warp_wait(pv_done(tl), (i - 1) & 1u, kSiteAttn + 10);
      if (!ok) break;
      tc_fence_after();
      const bool begins = w.unit == 0, ends = w.unit + static_cast<int>(end - begin) == w.units;
      const bool whole = begins && ends;
      const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (begins ? 1 : 0)) * kTileRows + 128 * tl + r;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t v[32];
        tmem_ld32(to + c, v);
        tmem_ld_wait(v);
        if (row.in && whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t o[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
              o[f] = pack_bf16x2(__uint_as_float(v[e + 2 * f]) * inv, __uint_as_float(v[e + 2 * f + 1]) * inv);
            stg8(p.o + row.at * kD + c + e, o);
          }
        } else if (row.in) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(ws.o + slot * kD + c + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        __syncwarp();
      }
      if (row.in) {
        if (!whole)
          ws.ml[slot] = make_float2(bs_row, l);
        else if (p.lse != nullptr)
          p.lse[row.at] = attn_lse(bs_row, l);
      }
      tc_fence_before();
      if (begins && !ends && tid == 0)
        ws.cut[blockIdx.x] = AttnCut{total, u0 + begin + w.units, w.b, w.hk, w.tile, 1};
      if (i < count) walk_item<kTileRows>(w, p, deal, places);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 11) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace coda
