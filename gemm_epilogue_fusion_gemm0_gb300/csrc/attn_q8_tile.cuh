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
// One block of 416 threads per SM:
//   warps 0..3, 4..7   softmax of tile 0, 1: a thread has a row (a lane of tensor memory), so a row's maximum
//                      and sum need no exchange.  S is read twice, for the maximum and for the exponentials: 128
//                      registers less than keeping it.
//   warps 8..11        widen k and v from global memory into shared memory, rings of two tiles each; a tile's
//                      codes are loaded to registers a unit ahead
//   warp 12            issues tcgen05.mma:  S_0(j + 1) behind P_0(j) v, S_1(j + 1) behind P_1(j) v, so that one tile's
//                      softmax runs beside the other's products
// o is rescaled only where a row's maximum has grown by more than 2^8 (P stays below fp16's largest): hardly ever
// after the first units.
#pragma once

#include "attn_q8.cuh"
#include "q8_mid.cuh"

namespace coda {

constexpr int kTileRows = 256, kTileThreads = 416;
constexpr int kTileStages = 2, kTileScales = 4;  // rings: of k's and v's tiles, of their scales
constexpr uint32_t kSiteAttn = 12;               // of bounded waits: kSiteAttn + which

template <int kD>
struct TileSmem {
  static constexpr uint32_t kOperand = 128 * kD * 2;  // 128 rows of fp16: panels of 64 columns
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kOperand;
  static constexpr uint32_t kV = kK + kTileStages * kOperand;
  static constexpr uint32_t kScale = kV + kTileStages * kOperand;  // [slot][k's 128, v's 128, 4 maxima of v's]
  static constexpr uint32_t kScaleSlot = 2 * 512 + 16;
  static constexpr uint32_t kBar = kScale + kTileScales * kScaleSlot;
  static constexpr uint32_t kBars = 4 * kTileStages + 2 * kTileScales + 8 + 1;
  static constexpr uint32_t kEnd = kBar + 8 * kBars;  // tensor memory's address, the abort flag
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

// 32 lanes x 16 columns: the thread's lane, columns [col, col + 16)
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

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

// The softmax's two walks over a row of S, 32 columns at a time with the next 32 on their way; `va` holds
// the first 32 between them.  `ts`: the thread's lane of S.  `sc`: k's 128 scales, then v's.
// kEdge: the row sees columns 0 .. seen only.
template <bool kEdge>
__device__ __forceinline__ void largest_of_32(const uint32_t (&v)[32], const float* sc, int seen, float& mx) {
  float m0 = mx, m1 = -INFINITY;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 k4 = *reinterpret_cast<const float4*>(sc + e);
    float x[4];
    unpack2(mul2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), pack2(k4.x, k4.y)), x[0], x[1]);
    unpack2(mul2(pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), pack2(k4.z, k4.w)), x[2], x[3]);
    if constexpr (kEdge) {
#pragma unroll
      for (int f = 0; f < 4; ++f)
        if (e + f > seen) x[f] = -INFINITY;
    }
    m0 = max3(m0, x[0], x[1]);
    m1 = max3(m1, x[2], x[3]);
  }
  mx = fmaxf(m0, m1);
}

template <bool kEdge>
__device__ __forceinline__ void largest_score(uint32_t ts, const float* sc, int seen, uint32_t (&va)[32],
                                              uint32_t (&vb)[32], float& mx) {
  tmem_ld32(ts, va);
  tmem_ld_wait(va);
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    tmem_ld32(ts + c + 32, vb);
    largest_of_32<kEdge>(va, sc + c, seen - c, mx);
    tmem_ld_wait(vb);
    tmem_ld32(ts + (c + 64) % 128, va);
    largest_of_32<kEdge>(vb, sc + c + 32, seen - c - 32, mx);
    tmem_ld_wait(va);
  }
}

// P = 2^(S k's scale rf - less) v's scale of 32 columns, in fp16 to tensor memory at `to`; the sum without v's.
template <bool kEdge>
__device__ __forceinline__ void weights_of_32(const uint32_t (&v)[32], const float* sc, int seen, uint64_t rf2,
                                              uint64_t less2, uint32_t to, uint64_t& sum2) {
  uint32_t pk[16];
  uint64_t sum[2] = {sum2, 0};
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 k4 = *reinterpret_cast<const float4*>(sc + e);
    const float4 v4 = *reinterpret_cast<const float4*>(sc + 128 + e);
    const uint64_t kk[2] = {pack2(k4.x, k4.y), pack2(k4.z, k4.w)};
    const uint64_t vv[2] = {pack2(v4.x, v4.y), pack2(v4.z, v4.w)};
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int at = e + 2 * f;
      const uint64_t x = mul2(pack2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), kk[f]);
      float a, b;
      unpack2(fma2(x, rf2, less2), a, b);
      a = ex2(a);
      b = ex2(b);
      if constexpr (kEdge) {
        if (at > seen) a = 0.f;
        if (at + 1 > seen) b = 0.f;
      }
      const uint64_t y = pack2(a, b);
      sum[f] = add2(sum[f], y);
      unpack2(mul2(y, vv[f]), a, b);
      if constexpr (kEdge) {  // (a scale behind the row's last key may be NaN)
        if (at > seen) a = 0.f;
        if (at + 1 > seen) b = 0.f;
      }
      pk[at / 2] = pack_f16x2(a, b);
    }
  }
  sum2 = add2(sum[0], sum[1]);
  tmem_st16(to, pk);  // (over columns of S that have been read)
}

template <bool kEdge>
__device__ __forceinline__ void weights(uint32_t ts, const float* sc, int seen, uint64_t rf2, uint64_t less2,
                                        uint32_t (&va)[32], uint32_t (&vb)[32], uint64_t& sum2) {
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    tmem_ld32(ts + c + 32, vb);
    weights_of_32<kEdge>(va, sc + c, seen - c, rf2, less2, ts + c / 2, sum2);
    tmem_ld_wait(vb);
    if (c == 0) tmem_ld32(ts + 64, va);
    weights_of_32<kEdge>(vb, sc + c + 32, seen - c - 32, rf2, less2, ts + c / 2 + 16, sum2);
    tmem_ld_wait(va);
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
      mbar_init(k_full(s), 4);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), 4);
      mbar_init(v_empty(s), 1);
    }
    for (uint32_t s = 0; s < kTileScales; ++s) {
      mbar_init(sc_full(s), 4);
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
  if (warp == 12) {
    tmem_alloc(base + Smem::kEnd, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + Smem::kEnd);
  const uint32_t count = static_cast<uint32_t>(u1 - u0);

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------- widening
    constexpr int kGroups = kD / 16;          // 16 codes each
    constexpr int kPer = 128 * kGroups / 128;  // of a thread and tensor
    const int pt = tid - 256;
    // Its 16 codes c of the rows r0 + i * 128 / kGroups.  The eight threads that write together have four
    // neighbouring groups of two rows: with the swizzle, 128 bytes without a bank twice.
    const uint32_t c = (pt & 3) + (kD == 128 ? 4 * ((pt >> 5) & 1) : 0);
    const uint32_t r0 = kD == 128 ? ((pt >> 2) & 7) + 8 * (pt >> 6) : pt >> 2;
    uint4 kr[kPer], vr[kPer];
    float ks = 0.f, vs = 0.f;
    // pages of the 8 groups of 16 keys of a unit, one per lane 0..7: looked up a unit before its loads
    const auto pages_at = [&](const AttnWalk& a) {
      const int key = a.unit * kAttnUnit + 16 * (lane & 7);
      return key < a.extent ? page_of(p.batch, p.cache, a.b, key) : -1;
    };
    const int mask = (1 << p.cache.page_log2) - 1;
    int pages = pages_at(w), pages_next = -1, key0 = 0, extent = 0, hk = 0;  // of the unit that is loaded
    uint32_t walked = 0;
    const auto next = [&]() {  // takes over the unit that `w` is at, and moves w to the one behind it
      key0 = w.unit * kAttnUnit;
      extent = w.extent;
      hk = w.hk;
      if (++walked < count) {
        walk_on<kTileRows>(w, p, deal, places);
        pages_next = pages_at(w);
      }
    };
    next();
    const auto load = [&](const uint8_t* q, uint4 (&to)[kPer]) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = static_cast<int>(r0) + i * (128 / kGroups);
        const int page = __shfl_sync(0xffffffffu, pages, r >> 4);
        to[i] = make_uint4(0u, 0u, 0u, 0u);
        if (page >= 0) {
          const size_t e = cache_entry(p.cache, page, hk, (key0 + r) & mask);
          to[i] = *reinterpret_cast<const uint4*>(q + e * kD + 16 * c);
        }
      }
    };
    const auto load_scales = [&]() {
      const int page = __shfl_sync(0xffffffffu, pages, pt >> 4), key = key0 + pt;
      ks = vs = key < extent ? __int_as_float(0x7fffffff) : 0.f;  // a page that does not exist: NaN
      if (page >= 0 && key < extent) {
        const size_t e = cache_entry(p.cache, page, hk, key & mask);
        ks = p.cache.k_s[e];
        vs = p.cache.v_s[e];
      }
    };
    const auto widen = [&](const uint4 (&from)[kPer], uint32_t to) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t r = r0 + i * (128 / kGroups);
        uint32_t x[8];
        q8_to_f16x2(from[i].x, x[0], x[1]);
        q8_to_f16x2(from[i].y, x[2], x[3]);
        q8_to_f16x2(from[i].z, x[4], x[5]);
        q8_to_f16x2(from[i].w, x[6], x[7]);
        st_shared_v4(to + panel_at(r, 2 * c), x[0], x[1], x[2], x[3]);
        st_shared_v4(to + panel_at(r, 2 * c + 1), x[4], x[5], x[6], x[7]);
      }
    };
    load_scales();
    load(p.cache.k_q, kr);
    load(p.cache.v_q, vr);
    for (uint32_t i = 0; i < count; ++i) {
      const uint32_t st = i % kTileStages, ph = i / kTileStages & 1u;
      const uint32_t sl = i % kTileScales, sph = i / kTileScales & 1u;
      if (!warp_wait(sc_empty(sl), sph ^ 1u, kSiteAttn)) break;
      float* const sc = reinterpret_cast<float*>(smem + Smem::kScale + sl * Smem::kScaleSlot);
      sc[pt] = ks;
      sc[128 + pt] = vs;
      const uint32_t vbits = fabsf(vs) <= 3.402823466e38f ? __float_as_uint(fabsf(vs)) : 0u;
      const uint32_t vmax = __reduce_max_sync(0xffffffffu, vbits);
      if (lane == 0) sc[256 + warp - 8] = __uint_as_float(vmax);
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_full(sl));
      if (!warp_wait(k_empty(st), ph ^ 1u, kSiteAttn + 1)) break;
      widen(kr, base + Smem::kK + st * Smem::kOperand);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(st));
      const bool more = i + 1 < count;
      if (more) {
        pages = pages_next;
        next();
        load_scales();
        load(p.cache.k_q, kr);
      }
      if (!warp_wait(v_empty(st), ph ^ 1u, kSiteAttn + 2)) break;
      widen(vr, base + Smem::kV + st * Smem::kOperand);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
      if (more) load(p.cache.v_q, vr);
    }
  } else if (warp == 12) {
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
    const float* const scales = reinterpret_cast<const float*>(smem + Smem::kScale);
    uint32_t i = 0;
    bool ok = true;
    while (ok && i < count) {
      // an item, or what of it lies in this block's share: its row of q, in fp16
      const uint32_t begin = i, end = i + min(static_cast<uint32_t>(w.units - w.unit), count - i);
      const AttnRow row = attn_row(p, w.s, w.hk, w.tile * kTileRows + static_cast<int>(128 * tl + r));
      const int limit = row.limit, low = __shfl_sync(0xffffffffu, limit, 0);  // (the smallest of the warp's rows)
      float rf;
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
        rf = p.scale_log2 * down;
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
      float m = -INFINITY, bs = -INFINITY, l = 0.f, lv = kLeastScale;
      int key = w.unit * kAttnUnit;
      for (; i < end; ++i, key += kAttnUnit) {
        const uint32_t uph = i & 1u, sl = i % kTileScales;
        ok = warp_wait(sc_full(sl), i / kTileScales & 1u, kSiteAttn + 8) && warp_wait(s_full(tl), uph, kSiteAttn + 9);
        if (!ok) break;
        tc_fence_after();
        const float* const sc = scales + sl * (Smem::kScaleSlot / 4);
        const bool edge = key + kAttnUnit - 1 > low;
        // The row's largest score.  The next 32 columns are on their way while 32 are looked at.
        const int seen = limit - key;  // columns 0 .. seen
        float mx = -INFINITY;
        uint32_t va[32], vb[32];
        if (edge)
          largest_score<true>(ts, sc, seen, va, vb, mx);
        else
          largest_score<false>(ts, sc, seen, va, vb, mx);
        const float4 vm = *reinterpret_cast<const float4*>(sc + 256);
        lv = fmaxf(lv, scale_power(fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w))));
        m = fmaxf(m, mx == -INFINITY ? mx : mx * rf);
        // what is taken out of the exponents: moved where P would leave fp16
        const bool move = m + lv > bs + 8.0f;
        if (__any_sync(0xffffffffu, move)) {
          const float corr = move ? ex2(bs - (m + lv)) : 1.0f;
          if (move) bs = m + lv;
          l *= corr;
          if (i > begin) {
            ok = warp_wait(pv_done(tl), uph ^ 1u, kSiteAttn + 10);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              tmem_ld32(to + c, vb);
              tmem_ld_wait(vb);
#pragma unroll
              for (int e = 0; e < 32; ++e) vb[e] = __float_as_uint(__uint_as_float(vb[e]) * corr);
              tmem_st32(to + c, vb);
            }
            tmem_st_wait();
          }
        }
        const float less = bs == -INFINITY ? 0.f : bs;  // (no key seen yet)
        uint64_t sum2 = 0;
        if (edge)
          weights<true>(ts, sc, seen, pack2(rf, rf), pack2(-less, -less), va, vb, sum2);
        else
          weights<false>(ts, sc, seen, pack2(rf, rf), pack2(-less, -less), va, vb, sum2);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_full(tl));
          mbar_arrive(sc_empty(sl));
        }
        float s0, s1;
        unpack2(sum2, s0, s1);
        l += s0 + s1;
      }
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
          ws.ml[slot] = make_float2(bs, l);
        else if (p.lse != nullptr)
          p.lse[row.at] = attn_lse(bs, l);
      }
      tc_fence_before();
      if (begins && !ends && tid == 0)
        ws.cut[blockIdx.x] = AttnCut{total, u0 + begin + w.units, w.b, w.hk, w.tile, 1};
      if (i < count) walk_item<kTileRows>(w, p, deal, places);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace coda
