// attn_q8_tile.cuh -- attention over the 8-bit paged cache for many rows (chunks and whole prompts): tiles of
// 256 packed rows on tcgen05.
//
// A block holds two tiles of 128 rows of q (fp16, shared memory) and walks the keys 128 at a time:
//   S_w = q_w k^T     128 x 128, tensor memory, fp32     (w = 0, 1: the two tiles)
//   P_w = 2^(S_w scale - base) * v's scale / power, fp16, over the first half of S_w's columns of the same keys
//   o_w += P_w v      128 x D, tensor memory; P_w is the first operand, from tensor memory
// in two halves of 64 keys each, so that a tile's softmax has one half to work at while the products of the other
// run (with all 128 together it waited for them: 4900 cycles a unit, of which the softmax was 2800).
// The tensor cores see codes widened to fp16 (exact); k's scales multiply S's columns and v's P's, in the softmax.
// Products are 4 * 256 * 128 * D operations per unit, 2048 cycles for D = 128.  Bound by shared memory: per unit 2048
// cycles of operands (S's 64 columns at a time read q again), 1024 of scales to the softmax, 1024 of codes in, read and
// widened out, 600 of the rest; measured 4300 to 5500 a unit with the pieces' ends.  A prompt of 8192 tokens of 32 heads of
// 128: 582 us, 0.94 PFLOP/s.
//
// One block of 704 threads per SM:
//   warps 0..7, 8..15  softmax of tile 0, 1: a warp has 16 rows, a thread 16 columns of a half of two of them.  (Four
//                      such warps to a quarter of the SM: the steps of an exponential depend on one another, and one
//                      warp alone takes 660 cycles for 32 of them in 32 lanes, two 740, four 1100.)
//   warps 16..19       widen k and v: codes from a ring that bulk copies fill, fp16 to the rings of two tiles each that
//                      the products read.  (With codes loaded to registers a unit ahead, by these warps, the softmax had
//                      none to keep its steps in flight; asked for by these warps, five copies a unit took each
//                      of them 2350 cycles.)
//   warp 20            issues tcgen05.mma: of each half of each tile, P v of a unit, then S of the next
//   warp 21            looks up pages, asks for their codes and puts a unit's scales into shared memory
// o is rescaled only where a row's maximum has grown by more than 2^8 or the largest of v's scales that it sees by a power
// of two (P stays below fp16's largest): hardly ever after the first units.
#pragma once

#include "attn_q8.cuh"
#include "q8_mid.cuh"

namespace coda {

constexpr int kTileStages = 2, kTileScales = 4;  // rings: of k's and v's tiles, of their scales
static_assert(kTileStages == 2, "the stage behind one is the other");
constexpr int kRawStages = 3;                    // ring of halves of a unit's codes (64 keys of k or v)
constexpr int kWideners = 4;                     // warps: 16 keys of a half each
constexpr uint32_t kSiteAttn = 12;               // of bounded waits: kSiteAttn + which

template <int kD>
struct TileSmem {
  static constexpr uint32_t kOperand = 128 * kD * 2;  // 128 rows of fp16: panels of 64 columns
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kOperand;
  static constexpr uint32_t kV = kK + kTileStages * kOperand;
  // [slot][k's 128, v's 128 divided by the power, v's 128, the power: of the largest of v's of the piece so far]
  static constexpr uint32_t kScale = kV + kTileStages * kOperand;
  static constexpr uint32_t kScaleSlot = 3 * 512 + 16;
  static constexpr uint32_t kRawBytes = 64 * kD;
  static constexpr uint32_t kRaw = (kScale + kTileScales * kScaleSlot + 127) / 128 * 128;
  static constexpr uint32_t kBar = kRaw + kRawStages * kRawBytes;
  static constexpr uint32_t kBars = 4 * kTileStages + 2 * kTileScales + 14 + 1 + 2 * kRawStages;
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

// A warp's 16 lanes x 64 columns of tensor memory: thread (g, t) has columns 8 i + 2 t, 8 i + 2 t + 1 of lane g in
// v[4 i], v[4 i + 1] and of lane g + 8 in v[4 i + 2], v[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// The same for 32 columns.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// 16 lanes x 32 columns: thread (g, t) writes column 4 i + t of lane g from v[2 i] and of lane g + 8 from v[2 i + 1].
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// What other threads wrote to shared memory before a barrier is seen by the tensor cores.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Where the 16-byte group c (8 values) of a row sits in an operand of panels of 64 columns, 128-byte
// swizzle: the layout of both the K-major operands (q, k) and the one whose rows are k (v).
__device__ __forceinline__ uint32_t panel_at(uint32_t row, uint32_t c) {
  return (c >> 3) * 16384u + row * 128u + (((c & 7u) ^ (row & 7u)) << 4);
}

// The softmax of 64 columns of a warp's 16 rows.  A thread has 16 columns of two rows, so a column's scale, read
// once, serves two products (with a row to a thread, the reads of scales alone took as long on shared memory as the
// operands of the products).  `sc`: k's scales (v's 128 and 256 numbers on) from the thread's first column.
// kEdge: row k sees columns 0 .. seen[k] of those from there on, and has a power of its own.

// S times k's scales, and its largest.
template <bool kEdge>
__device__ __forceinline__ void scaled(uint32_t (&v)[32], const float* sc, const int (&seen)[2], float (&mx)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 k2 = *reinterpret_cast<const float2*>(sc + 8 * i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x, y;
      unpack2(mul2(pack2(__uint_as_float(v[4 * i + 2 * k]), __uint_as_float(v[4 * i + 2 * k + 1])), pack2(k2.x, k2.y)),
              x, y);
      if constexpr (kEdge) {
        if (8 * i > seen[k]) x = -INFINITY;
        if (8 * i + 1 > seen[k]) y = -INFINITY;
      }
      mx[k] = max3(mx[k], x, y);
      v[4 * i + 2 * k] = __float_as_uint(x);
      v[4 * i + 2 * k + 1] = __float_as_uint(y);
    }
  }
}

// P = 2^(what `scaled` left * rf - less) v's scale / power in fp16; the sums without these two.
template <bool kEdge>
__device__ __forceinline__ void weights(const uint32_t (&v)[32], const float* sc, const int (&seen)[2], const float (&rf)[2],
                                        const float (&less)[2], const float (&power)[2], uint32_t (&pk)[16],
                                        uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 v2 = *reinterpret_cast<const float2*>(sc + (kEdge ? 256 : 128) + 8 * i);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x, y;
      unpack2(fma2(pack2(__uint_as_float(v[4 * i + 2 * k]), __uint_as_float(v[4 * i + 2 * k + 1])), pack2(rf[k], rf[k]),
                   pack2(-less[k], -less[k])),
              x, y);
      x = ex2(x);
      y = ex2(y);
      if constexpr (kEdge) {
        if (8 * i > seen[k]) x = 0.f;
        if (8 * i + 1 > seen[k]) y = 0.f;
      }
      const uint64_t xy = pack2(x, y);
      sum[k] = add2(sum[k], xy);
      if constexpr (kEdge) {
        const float by = power_inverse(power[k]);
        unpack2(mul2(xy, mul2(pack2(v2.x, v2.y), pack2(by, by))), x, y);
      } else {
        unpack2(mul2(xy, pack2(v2.x, v2.y)), x, y);
      }
      if constexpr (kEdge) {  // (a scale behind the row's last key may be NaN)
        if (8 * i > seen[k]) x = 0.f;
        if (8 * i + 1 > seen[k]) y = 0.f;
      }
      pk[2 * i + k] = pack_f16x2(x, y);
    }
  }
}

// o of a warp's rows, two of the thread's, times a number each.  (Not inlined: hardly ever called.)
template <int kD>
__device__ __noinline__ void rescale_rows(uint32_t to, float by0, float by1) {
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < kD; c += 32) {
    uint32_t o[16];
    tmem_ld_16x32(to + c, o);
    tmem_ld_wait(o);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (e >> 1 & 1 ? by1 : by0));
    tmem_st_16x256b_x4(to + c, o);
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
  // w: 2 * tile + half of the unit's keys
  const auto s_full = [&](uint32_t w) { return bars + 8u * (kB + w); };       // S is there
  const auto p_full = [&](uint32_t w) { return bars + 8u * (kB + 4 + w); };   // P is there
  const auto pv_done = [&](uint32_t w) { return bars + 8u * (kB + 8 + w); };  // o has P v
  const auto q_full = [&](uint32_t t) { return bars + 8u * (kB + 12 + t); };
  const uint32_t drained = bars + 8u * (kB + 14);
  const auto raw_full = [&](uint32_t i) { return bars + 8u * (kB + 15 + i); };
  const auto raw_empty = [&](uint32_t i) { return bars + 8u * (kB + 15 + kRawStages + i); };
  volatile uint32_t* const abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Smem::kEnd + 4);
  const WaitCtl wc{timeout_ns, &g_coda_status, abort_flag};
  // a whole warp waits, and gives up, together
  const auto warp_wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, wc, site)) != 0;
  };
  griddep_launch_dependents();
  griddep_wait();

  AttnWalk w;
  int64_t end;
  bool some;
  const int64_t total = walk_start<TileDeal>(w, p, deal, places, reinterpret_cast<int64_t*>(smem), end, some);
  if (tid == 0) ws.cut[blockIdx.x].cut.valid = 0;
  // (the first piece; each role walks the others by itself)
  if (!some || !walk_piece<TileDeal>(w, p, deal, places)) return;
  if (tid == 0) {
    *abort_flag = 0u;
    for (uint32_t s = 0; s < kTileStages; ++s) {
      mbar_init(k_full(s), kWideners);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), kWideners);
      mbar_init(v_empty(s), 1);
    }
    for (uint32_t s = 0; s < kTileScales; ++s) {
      mbar_init(sc_full(s), 1);
      mbar_init(sc_empty(s), 16);
    }
    for (uint32_t i = 0; i < 4; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 8);
      mbar_init(pv_done(i), 1);
    }
    for (uint32_t i = 0; i < 2; ++i) mbar_init(q_full(i), 8);
    mbar_init(drained, 1);
    for (uint32_t i = 0; i < kRawStages; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), kWideners);
    }
    fence_mbar_init();
  }
  if (warp == 20) {
    tmem_alloc(base + Smem::kEnd, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (from one lane: known to be the same in the whole warp)
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + Smem::kEnd), 0);

  if (warp >= 16 && warp < 20) {
    // ------------------------------------------------------------- widening
    constexpr int kPer = kD / 32;  // of a lane and half, 16 codes each
    const uint32_t mine = static_cast<uint32_t>(warp - 16);  // its 16 keys of a half
    // The lane's j-th 16 codes: eight lanes have four of one key and the other four of the next, which are
    // 128 bytes without a bank twice both where they are read and, with the swizzle, where they go.
    const uint32_t q = lane & 7;
    const auto row_at = [&](int j) {
      return 16u * mine + (kD == 128 ? 2u * (lane >> 3) + (q >> 2) + 8u * (j >> 1) : static_cast<uint32_t>(lane >> 2) + 8u * j);
    };
    const auto col_at = [&](int j) { return kD == 128 ? q ^ (4u * (j & 1)) : q & 3u; };
    uint32_t half = 0;  // halves done
    const auto widen = [&](uint32_t to) {
      const uint32_t slot = half % kRawStages;
      if (!warp_wait(raw_full(slot), half / kRawStages & 1u, kSiteAttn + 12)) return false;
      ++half;
      uint4 x[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        x[j] = ld_shared_v4(base + Smem::kRaw + slot * Smem::kRawBytes + row_at(j) * kD + 16u * col_at(j));
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const uint32_t r = row_at(j), c = 2u * col_at(j);
        uint32_t y[8];
        q8_to_f16x2(x[j].x, y[0], y[1]);
        q8_to_f16x2(x[j].y, y[2], y[3]);
        q8_to_f16x2(x[j].z, y[4], y[5]);
        q8_to_f16x2(x[j].w, y[6], y[7]);
        st_shared_v4(to + panel_at(r, c), y[0], y[1], y[2], y[3]);
        st_shared_v4(to + panel_at(r, c + 1u), y[4], y[5], y[6], y[7]);
      }
      // Behind the last use of what was read: the barrier does not wait for a read in flight, and a copy that came
      // in between was seen to change it (half of the calls of one shape).
      __syncwarp();
      if (lane == 0) mbar_arrive(raw_empty(slot));
      return true;
    };
    for (uint32_t i = 0; i == 0 || walk_unit<TileDeal>(w, p, deal, places); ++i) {
      const uint32_t st = i % kTileStages, ph = i / kTileStages & 1u;
      const uint32_t k = base + Smem::kK + st * Smem::kOperand, v = base + Smem::kV + st * Smem::kOperand;
      if (!warp_wait(k_empty(st), ph ^ 1u, kSiteAttn + 1) || !widen(k) || !widen(k + 64 * 128)) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(k_full(st));
      if (!warp_wait(v_empty(st), ph ^ 1u, kSiteAttn + 2) || !widen(v) || !widen(v + 64 * 128)) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
    }
  } else if (warp == 21) {
    // ------------------------------------------------------------- pages, copies, scales
    // A copy takes as many keys as lie together, `keys`: a page's, 64 at most.
    const int keys = min(1 << p.cache.page_log2, 64), log2 = min(p.cache.page_log2, 6);
    const int mask = (1 << p.cache.page_log2) - 1;
    // the table's entry for the lane's keys of a unit (lanes below 128 / keys): asked for a unit before it is used
    const auto entry_at = [&](const AttnWalk& a) {
      const int key = a.unit * kAttnUnit + lane * keys, i = key >> p.cache.page_log2;
      return key < a.extent && i < p.batch.width ? __ldg(p.batch.table + static_cast<size_t>(a.b) * p.batch.width + i) : -1;
    };
    int entry = entry_at(w);
    uint32_t half = 0;
    bool ok = true, more = true;
    float power = kLeastScale;  // of the largest scale of v so far in the piece
    for (uint32_t i = 0; more; ++i) {
      const int key0 = w.unit * kAttnUnit, extent = w.extent, hk = w.hk;
      const bool last = w.unit + 1 == w.last;  // of the piece
      const bool bad = static_cast<unsigned>(entry) >= static_cast<unsigned>(p.cache.pages);
      if (bad && lane < kAttnUnit / keys && key0 + lane * keys < extent) atomicCAS(&g_coda_status, 0u, 0x200u | kChkPage);
      const int page = bad ? -1 : entry;
      const size_t at = cache_entry(p.cache, max(page, 0), hk, (key0 + lane * keys) & mask) * kD;
      // its scales: of keys 4 lane .. 4 lane + 3
      const int spage = __shfl_sync(0xffffffffu, page, 4 * lane >> log2), skey = key0 + 4 * lane;
      const size_t se = cache_entry(p.cache, max(spage, 0), hk, skey & mask);
      float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
      if (entries_ok(p.cache, se, 4)) {
        ks = *reinterpret_cast<const float4*>(p.cache.k_s + se);
        vs = *reinterpret_cast<const float4*>(p.cache.v_s + se);
      }
      // The codes of 64 keys; where there are none (behind the last key, or a page that does not exist) any will do:
      // their scales are zero or NaN.
      const auto ask = [&](const uint8_t* codes, int h) {
        const uint32_t slot = half % kRawStages;
        if (!warp_wait(raw_empty(slot), (half / kRawStages & 1u) ^ 1u, kSiteAttn + 13)) return false;
        ++half;
        const bool mine = page >= 0 && lane >> (6 - log2) == h && entries_ok(p.cache, at / kD, keys);
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, mine));
        const uint32_t bytes = static_cast<uint32_t>(keys) * kD;
        if (lane == 0) {
          if (copies > 0)
            mbar_arrive_expect_tx(raw_full(slot), copies * bytes);
          else
            mbar_arrive(raw_full(slot));
        }
        __syncwarp();
        if (mine)
          bulk_load(base + Smem::kRaw + slot * Smem::kRawBytes + static_cast<uint32_t>(lane - (h << (6 - log2))) * bytes,
                    codes + at, bytes, raw_full(slot));
        __syncwarp();
        return true;
      };
      ok = ask(p.cache.k_q, 0) && ask(p.cache.k_q, 1);
      if (!ok) break;
      more = walk_unit<TileDeal>(w, p, deal, places);
      if (more) entry = entry_at(w);
      const auto given = [&](float s, int e) {  // nothing behind the last key is looked at; NaN for a page that does not exist
        return skey + e >= extent ? 0.f : spage < 0 ? __int_as_float(0x7fffffff) : s;
      };
      const float part = p.scale_part;
      ks = make_float4(given(ks.x, 0) * part, given(ks.y, 1) * part, given(ks.z, 2) * part, given(ks.w, 3) * part);
      vs = make_float4(given(vs.x, 0), given(vs.y, 1), given(vs.z, 2), given(vs.w, 3));
      const uint32_t sl = i % kTileScales;
      ok = warp_wait(sc_empty(sl), (i / kTileScales & 1u) ^ 1u, kSiteAttn);
      if (!ok) break;
      float* const sc = reinterpret_cast<float*>(smem + Smem::kScale + sl * Smem::kScaleSlot);
      const float top = fmaxf(fmaxf(finite_size(vs.x), finite_size(vs.y)), fmaxf(finite_size(vs.z), finite_size(vs.w)));
      const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      power = fmaxf(power, scale_power(__uint_as_float(all)));
      const float by = power_inverse(power);
      *reinterpret_cast<float4*>(sc + 4 * lane) = ks;
      *reinterpret_cast<float4*>(sc + 128 + 4 * lane) = make_float4(vs.x * by, vs.y * by, vs.z * by, vs.w * by);
      *reinterpret_cast<float4*>(sc + 256 + 4 * lane) = vs;
      if (lane == 0) sc[384] = power;
      if (last) power = kLeastScale;
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_full(sl));
      ok = ask(p.cache.v_q, 0) && ask(p.cache.v_q, 1);
      if (!ok) break;
    }
    // (also where a wait ran out: no copy is in flight when the block leaves)
    if (lane == 0) land_copies(raw_full(0), static_cast<int>(half), kRawStages, timeout_ns);
  } else if (warp == 20) {
    // ------------------------------------------------------------- products
    const bool issuer = elect_one();
    constexpr uint32_t kIdescS = idesc_f16_f32(128, 64);
    constexpr uint32_t kIdescO = idesc_f16_f32(128, kD) | (1u << 16);  // v: rows are k
    // Descriptors are sums of constants and of what is known to be the same in the whole warp (`stage`: from one
    // lane), so that an instruction's operands are in uniform registers: 60 cycles each where they were not.
    const uint64_t dq = sdesc_sw128(base + Smem::kQ, 16, 1024), dk = sdesc_sw128(base + Smem::kK, 16, 1024);
    const uint64_t dv = sdesc_sw128(base + Smem::kV, 16384, 1024);
    const auto stage = [&](uint32_t i) { return __shfl_sync(0xffffffffu, i % kTileStages, 0); };
    const auto s_mma = [&](uint32_t t, uint32_t h, uint32_t st) {
      const uint64_t a = dq + t * (Smem::kOperand >> 4), b = dk + st * (Smem::kOperand >> 4) + h * (8192u >> 4);
#pragma unroll
      for (uint32_t k = 0; k < kD / 16; ++k) {
        const uint32_t off = ((k / 4) * 16384u + (k % 4) * 32u) >> 4;
        if (issuer) umma_bf16(tmem + 128u * t + 64u * h, a + off, b + off, kIdescS, k > 0);
      }
      if (issuer) umma_commit(s_full(2 * t + h));
    };
    const auto o_mma = [&](uint32_t t, uint32_t h, uint32_t st, bool first) {
      const uint64_t b = dv + st * (Smem::kOperand >> 4) + h * (8192u >> 4);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        if (issuer)
          umma_f16_ts(tmem + 256u + kD * t, tmem + 128u * t + 64u * h + 8u * k, b + k * (2048u >> 4), kIdescO,
                      !first || k > 0);
      if (issuer) umma_commit(pv_done(2 * t + h));
    };
    const auto wait_all = [&](uint32_t bar, uint32_t parity, uint32_t site) {
      const bool ok = warp_wait(bar, parity, site);
      tc_fence_after();
      return ok;
    };
    uint32_t i = 0;
    bool ok = true;
    for (uint32_t pieces = 0; pieces == 0 || walk_piece<TileDeal>(w, p, deal, places); ++pieces) {
      const uint32_t stop = i + static_cast<uint32_t>(w.last - w.unit);
      uint32_t st = stage(i);
      ok = wait_all(q_full(0), pieces & 1u, kSiteAttn + 3) && wait_all(q_full(1), pieces & 1u, kSiteAttn + 3) &&
           wait_all(k_full(st), i / kTileStages & 1u, kSiteAttn + 4);
      if (!ok) break;
#pragma unroll
      for (uint32_t w4 = 0; w4 < 4; ++w4) s_mma(w4 & 1, w4 >> 1, st);
      if (issuer) umma_commit(k_empty(st));
      for (bool first = true; i < stop; ++i, first = false) {
        st = stage(i);
        const uint32_t ph = i / kTileStages & 1u, uph = i & 1u;
        const uint32_t nst = st ^ 1u, nph = (i + 1) / kTileStages & 1u;
        const bool more = i + 1 < stop;
        ok = wait_all(v_full(st), ph, kSiteAttn + 5);
        if (!ok) break;
#pragma unroll
        for (uint32_t w4 = 0; w4 < 4; ++w4) {
          const uint32_t t = w4 & 1, h = w4 >> 1;
          ok = wait_all(p_full(2 * t + h), uph, kSiteAttn + 6);
          if (!ok) break;
          o_mma(t, h, st, first && h == 0);
          if (w4 == 3 && issuer) umma_commit(v_empty(st));
          if (more) {
            if (w4 == 0) {
              ok = wait_all(k_full(nst), nph, kSiteAttn + 4);
              if (!ok) break;
            }
            s_mma(t, h, nst);
            if (w4 == 3 && issuer) umma_commit(k_empty(nst));
          }
        }
        if (!ok) break;
      }
      if (!ok) break;
    }
    // (no product is left in flight when the tensor memory is given back)
    if (issuer) umma_commit(drained);
    bounded_wait(drained, 0, wc, kSiteAttn + 7);
  } else if (warp < 16) {
    // ------------------------------------------------------------- softmax
    const uint32_t tl = static_cast<uint32_t>(warp) >> 3;
    const uint32_t r0 = 32u * (warp & 3) + 16u * (warp >> 2 & 1);  // its first row of the tile
    const uint32_t ts = tmem + 128u * tl + (r0 << 16), to = tmem + 256u + kD * tl + (r0 << 16);
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    const float* const scales = reinterpret_cast<const float*>(smem + Smem::kScale);
    uint32_t i = 0;
    bool ok = true;
    do {
      // a piece of an item
      const uint32_t begin = i, stop = i + static_cast<uint32_t>(w.last - w.unit);
      const int packed = w.tile * kTileRows + static_cast<int>(128 * tl + r0);
      float rf[2];
      {  // The rows of q, in fp16: D / 8 lanes read a row, so a read is whole rows.
        constexpr int kLanes = kD / 8, kPer = kD / 16;  // lanes of a row; reads, of 32 / kLanes rows each
        const int c = lane % kLanes, up_row = lane / kLanes;
        Chunk8 x[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const AttnRow row = attn_row(p, w.s, w.hk, packed + j * (32 / kLanes) + up_row);
          x[j] = Chunk8{{0u, 0u, 0u, 0u}};
          if (row_ok(p, row, kChkLoad)) x[j] = ldg8(p.q + row.at * kD + 8 * c);
        }
        float mine = 0.f;  // what row lane % 16 is multiplied by afterwards
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          float v[8], amax = 0.f;
          unpack8(x[j], v);
#pragma unroll
          for (int e = 0; e < 8; e += 2) amax = max3_abs_nan(amax, v[e], v[e + 1]);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          float up, down;
          row_power(amax, up, down);
          const float got = __shfl_sync(0xffffffffu, down, lane % (32 / kLanes) * kLanes);
          if ((lane & 15) / (32 / kLanes) == j) mine = got;
          st_shared_v4(base + Smem::kQ + tl * Smem::kOperand + panel_at(r0 + j * (32 / kLanes) + up_row, c),
                       pack_f16x2(v[0] * up, v[1] * up), pack_f16x2(v[2] * up, v[3] * up),
                       pack_f16x2(v[4] * up, v[5] * up), pack_f16x2(v[6] * up, v[7] * up));
        }
        mine = exponent_factor(p.scale_power, mine);
        rf[0] = __shfl_sync(0xffffffffu, mine, g);
        rf[1] = __shfl_sync(0xffffffffu, mine, g + 8);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(tl));
      const AttnRow row[2] = {attn_row(p, w.s, w.hk, packed + g), attn_row(p, w.s, w.hk, packed + g + 8)};
      const int low = __shfl_sync(0xffffffffu, row[0].limit, 0);  // the smallest of the warp's rows
      float bs[2];
      float power[2];  // of v's scales, in o
      uint64_t sum[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        power[k] = kLeastScale;
        bs[k] = -INFINITY;
        sum[k] = 0;
      }
      int key = w.unit * kAttnUnit;
      for (; ok && i < stop; ++i, key += kAttnUnit) {
        const uint32_t uph = i & 1u, sl = i % kTileScales;
        ok = warp_wait(sc_full(sl), i / kTileScales & 1u, kSiteAttn + 8);
        if (!ok) break;
        const float* const sc = scales + sl * (Smem::kScaleSlot / 4);
        const float given = sc[384];
        const bool edge = key + kAttnUnit - 1 > low;
        // (hardly ever after a piece's first units)
        if (__any_sync(0xffffffffu, given > power[0] || given > power[1])) {
          float corr[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float to_be = given;
            if (edge) {  // what its rows see alone
              const int seen = row[k].limit - (key + t2);
              float vm = 0.f;
#pragma unroll 1
              for (int c = 0; c < kAttnUnit; c += 8) {
                const float2 vs = *reinterpret_cast<const float2*>(sc + 256 + t2 + c);
                if (c <= seen) vm = fmaxf(vm, finite_size(vs.x));
                if (c + 1 <= seen) vm = fmaxf(vm, finite_size(vs.y));
              }
              vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
              vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
              to_be = fmaxf(power[k], scale_power(vm));
            }
            corr[k] = ex2(power_log2(power[k], to_be));
            power[k] = to_be;
          }
          if (i > begin) {
            ok = warp_wait(pv_done(2 * tl + 1), uph ^ 1u, kSiteAttn + 10);
            if (!ok) break;
            rescale_rows<kD>(to, corr[0], corr[1]);
          }
        }
#pragma unroll 1
        for (uint32_t h = 0; h < 2; ++h) {
          ok = warp_wait(s_full(2 * tl + h), uph, kSiteAttn + 9);
          if (!ok) break;
          tc_fence_after();
          const float* const hsc = sc + 64 * h + t2;
          const int before = t2 + key + 64 * static_cast<int>(h);
          const int seen[2] = {row[0].limit - before, row[1].limit - before};
          uint32_t v[32];
          tmem_ld_16x64(ts + 64u * h, v);
          tmem_ld_wait(v);
          float mx[2] = {-INFINITY, -INFINITY};
          if (edge)
            scaled<true>(v, hsc, seen, mx);
          else
            scaled<false>(v, hsc, seen, mx);
          // What is taken out of the exponents, and of the values' scales, moves where P would leave fp16: to the row's
          // largest score of these keys, and to the largest of their scales.
          const bool fits = mx[0] * rf[0] <= bs[0] + 8.0f && mx[1] * rf[1] <= bs[1] + 8.0f;
          if (!__all_sync(0xffffffffu, fits)) {
            bool move = false;
            float corr[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
              mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
              const float to_be = mx[k] == -INFINITY ? mx[k] : mx[k] * rf[k];
              corr[k] = 1.0f;
              if (to_be > bs[k] + 8.0f) {
                move = true;
                corr[k] = ex2(bs[k] - ceilf(to_be));
                bs[k] = ceilf(to_be);  // (a whole number: see the kernel for few)
              }
              sum[k] = mul2(sum[k], pack2(corr[k], corr[k]));
            }
            if ((i > begin || h > 0) && __any_sync(0xffffffffu, move)) {
              ok = warp_wait(pv_done(2 * tl + (h ^ 1u)), h == 0 ? uph ^ 1u : uph, kSiteAttn + 10);
              if (!ok) break;
              rescale_rows<kD>(to, corr[0], corr[1]);
            }
          }
          const float less[2] = {bs[0] == -INFINITY ? 0.f : bs[0], bs[1] == -INFINITY ? 0.f : bs[1]};  // (no key seen yet)
          uint32_t pk[16];
          if (edge)
            weights<true>(v, hsc, seen, rf, less, power, pk, sum);
          else
            weights<false>(v, hsc, seen, rf, less, power, pk, sum);
          tmem_st_16x128b_x8(ts + 64u * h, pk);  // over S, which is read
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(2 * tl + h));
        }
        if (ok && lane == 0) mbar_arrive(sc_empty(sl));
      }
      if (!ok) break;
      float l[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        unpack2(sum[k], x, y);
        x += y;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        l[k] = x + __shfl_xor_sync(0xffffffffu, x, 2);
      }
      // (a barrier for each half: with one for both, of which this waits for the second last phase's successor, the
      // wait took a phase further back for it)
      ok = warp_wait(pv_done(2 * tl), (i - 1) & 1u, kSiteAttn + 10) &&
           warp_wait(pv_done(2 * tl + 1), (i - 1) & 1u, kSiteAttn + 10);
      if (!ok) break;
      tc_fence_after();
      const bool whole = w.begins && w.ends;
      const size_t slot = (2 * static_cast<size_t>(blockIdx.x) + (w.begins ? 1 : 0)) * kTileRows + 128 * tl + r0;
      // The outputs go through the warp's rows of q's place, which the products have left, so that whole rows, or
      // 128 bytes of them in fp32, are written at a time.  (32 columns together: with 64 the loops' registers spill.)
      const uint32_t stage = base + Smem::kQ + tl * Smem::kOperand;
      const int in_rows = min(16, max(0, w.s.n * p.group - packed));
      // (the quotient within 2 ulp; no sum is near 2^126)
      const float by[2] = {l[0] == 0.f ? 0.f : __fdividef(power_unit(power[0]), l[0]),
                           l[1] == 0.f ? 0.f : __fdividef(power_unit(power[1]), l[1])};
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t v[16];
        tmem_ld_16x32(to + c, v);
        tmem_ld_wait(v);
        if (whole) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_shared_u32(stage + panel_at(r0 + g + 8 * k, c / 8 + j) + 2 * t2,
                            pack_bf16x2(__uint_as_float(v[4 * j + 2 * k]) * by[k], __uint_as_float(v[4 * j + 2 * k + 1]) * by[k]));
        } else {
          const auto place = [&](uint32_t r, uint32_t c16) {  // 16 rows of 128 bytes: the 16-byte group c16 of row r
            return stage + (r0 + r) * 128u + ((c16 ^ (r & 7u)) << 4);
          };
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t at = place(g + 8 * k, 2 * j + (t2 >> 2)) + 4 * (t2 & 2);
              st_shared_u32(at, v[4 * j + 2 * k]);
              st_shared_u32(at + 4, v[4 * j + 2 * k + 1]);
            }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 4 * j + (lane >> 3), c16 = lane & 7;
            if (r < in_rows && part_ok(ws, (slot + r) / kTileRows, static_cast<int>((slot + r) % kTileRows)))
              *reinterpret_cast<uint4*>(ws.o + (slot + r) * kD + c + 4 * c16) = ld_shared_v4(place(r, c16));
          }
          __syncwarp();
        }
      }
      if (whole) {
        __syncwarp();
        constexpr int kLanes = kD / 8;
#pragma unroll
        for (int j = 0; j < kD / 16; ++j) {
          const int r = j * (32 / kLanes) + lane / kLanes, c = lane % kLanes;
          if (r < in_rows) {
            const AttnRow at = attn_row(p, w.s, w.hk, packed + r);
            if (!row_ok(p, at, kChkStore)) continue;
            *reinterpret_cast<uint4*>(p.o + at.at * kD + 8 * c) = ld_shared_v4(stage + panel_at(r0 + r, c));
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (row[k].in && t2 == 0) {
          if (!whole) {
            if (!part_ok(ws, (slot + g + 8 * k) / kTileRows, static_cast<int>((slot + g + 8 * k) % kTileRows))) continue;
            ws.ml[slot + g + 8 * k] = make_float2(bs[k], l[k]);
            ws.unit[slot + g + 8 * k] = power_unit(power[k]);
          } else if (p.lse != nullptr && row_ok(p, row[k], kChkStore))
            p.lse[row[k].at] = attn_lse(bs[k], l[k]);
        }
      tc_fence_before();
      if (tid == 0) tell_cut(w, &ws.cut[blockIdx.x].cut, total, end);
    } while (walk_piece<TileDeal>(w, p, deal, places));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 20) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace coda
