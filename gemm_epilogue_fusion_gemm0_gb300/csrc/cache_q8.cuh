// cache_q8.cuh -- the 8-bit paged cache: writing a projection's rows into it and reading them back.
//
// The cache holds keys and values as INT8 codes with one fp32 scale per token and head, in pages of
// `page` tokens:  codes [pages, Hk, page, D],  scales [pages, Hk, page].  A sequence's tokens lie in
// the pages that its row of the table names, in order.  All operators take the same description of a
// batch: rows cu[b] .. cu[b + 1] - 1 are the last rows of sequence b's lens[b] tokens, so row i has
// the position lens[b] - (cu[b + 1] - i).
#pragma once

#include "q8_small.cuh"

namespace coda {

constexpr uint32_t kChkPage = 0x40;  // a page outside of the cache or of the table (every build)

struct CacheQ8 {
  uint8_t* k_q;
  float* k_s;
  uint8_t* v_q;
  float* v_s;
  int pages, page_log2, Hk;
};

struct BatchQ8 {
  const int32_t* cu;     // [B + 1]
  const int32_t* lens;   // [B]
  const int32_t* table;  // [B, width]
  int B, width;
  int rows;
};

// The page that holds position `pos` >= 0 of sequence b, or -1 (recorded) where the table has no
// such place or names a page that the cache does not have.
__device__ __forceinline__ int page_of(const BatchQ8& bt, const CacheQ8& c, int b, int pos) {
  const int i = pos >> c.page_log2;
  int page = -1;
  if (i < bt.width) page = __ldg(bt.table + static_cast<size_t>(b) * bt.width + i);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.pages)) {
    atomicCAS(&g_coda_status, 0u, 0x200u | kChkPage);
    return -1;
  }
  return page;
}

// First entry (token, head) of a page's slot: times D the codes' index, by itself the scale's.
__device__ __forceinline__ size_t cache_entry(const CacheQ8& c, int page, int head, int slot) {
  return ((static_cast<size_t>(page) * c.Hk + head) << c.page_log2) + slot;
}

// n entries from e on, of the cache (in the checked build)
__device__ __forceinline__ bool entries_ok(const CacheQ8& c, size_t e, int n) {
  return checked(e + n <= (static_cast<size_t>(c.pages) * c.Hk) << c.page_log2, kChkCache);
}
// head h of `heads` of a row of the call
__device__ __forceinline__ bool head_ok(const BatchQ8& bt, size_t row, int h, int heads, uint32_t site) {
  return checked(row < static_cast<size_t>(bt.rows) && h >= 0 && h < heads, site);
}

// The sequence that a row belongs to, by a whole warp: the count of b in 1 .. B with cu[b] <= row.
// 32 bounds at a time, so two loads one after the other serve 1024 sequences.  B for a row behind the
// last sequence.
__device__ __forceinline__ int sequence_of(const BatchQ8& bt, int row, int lane) {
  int lo = 0, hi = bt.B;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool before = at <= hi && __ldg(bt.cu + at) <= row;
    lo += __popc(__ballot_sync(0xffffffffu, before)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// A row's place.
struct RowPlace {
  int seq;   // -1: the row belongs to no sequence
  int pos;   // its position (negative: it stands before its sequence's first token)
  int page;  // -1: none
  int slot;
};

__device__ __forceinline__ RowPlace place_of(const BatchQ8& bt, const CacheQ8& c, int row, int lane) {
  RowPlace p = {-1, 0, -1, 0};
  if (row >= bt.rows) return p;
  const int b = sequence_of(bt, row, lane);
  if (b >= bt.B || row < __ldg(bt.cu)) return p;
  p.seq = b;
  p.pos = __ldg(bt.lens + b) - (__ldg(bt.cu + b + 1) - row);
  if (p.pos < 0) return p;
  p.page = page_of(bt, c, b, p.pos);
  p.slot = p.pos & ((1 << c.page_log2) - 1);
  return p;
}

// ---------------------------------------------------------------------------
// Write: y's row of a token holds Hq + 2 Hk heads [q | k | v].  The first 2 * half values of a head of
// q and k are turned in pairs (a, b):
//   a' = a cos - b sin,  b' = a sin + b cos,  angle = pos[axis(i)] * inv_freq(i)
// pair i being values (i, i + half), or (2 i, 2 i + 1).  q goes out in bf16; k (after its turn, in
// fp32) and v become codes.
//
// Angles: a turn is 2^64, turn[i] = inv_freq / (2 pi) of it, and the product with the position modulo
// 2^64 is the angle's fraction of a turn to |pos| 2^-64 of a turn (frequencies up to 2^40), whatever the number of
// turns: no position is too far.  Its upper 32 bits go, rounded to fp32 (2^-26 of a turn, 1.6 ulp of an fp32 sine
// or cosine near one at most), to sincospif (2 ulp).
//
// Bound by HBM: 2 (Hq + 2 Hk) D bytes in, 2 Hq D + 2 Hk (D + 4) out per token.  A block takes kTokens
// tokens: its threads find the tokens' places and form their angles' cos and sin once, one each, then D / 8
// threads share a head (16 bytes in each), and a group of them walks the heads of one token, kWriteBatch at a
// time: their loads go out together, the first ones before the places are known.  (One head at a time, with the
// shuffles of its maximum between the loads: 83 us for 8192 tokens of 64 + 16 heads of 128.)
// ---------------------------------------------------------------------------
constexpr int kRopeMax = 64;  // pairs
constexpr int kRopeAxes = 4;

struct RopeQ8 {
  uint64_t turn[kRopeMax];
  uint8_t axis[kRopeMax];
  const int32_t* pos;  // [axes, rows], or null: the token's position in its sequence
  int half;            // pairs; 0: no turn
  int pairs;           // 1: neighbours
};

struct CacheWriteParams {
  const __nv_bfloat16* y;
  __nv_bfloat16* q_out;
  CacheQ8 cache;
  BatchQ8 batch;
  int Hq;
};

constexpr int kCacheThreads = 256;
constexpr int kWriteBatch = 5;

template <int kD, int kTokens>
__global__ void __launch_bounds__(kCacheThreads, 3)
    cache_write_q8_kernel(const CacheWriteParams p, const __grid_constant__ RopeQ8 rope) {
  constexpr int kLanes = kD / 8;                            // threads per head
  constexpr int kGroups = kCacheThreads / kLanes / kTokens;  // heads of a token at a time
  __shared__ RowPlace place[kTokens];
  __shared__ float cs[kTokens][kRopeMax], sn[kTokens][kRopeMax];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int row0 = static_cast<int>(blockIdx.x) * kTokens;
  const int group = tid / kLanes, c = tid % kLanes;  // c: this thread's 8 values of the head
  const int t = group / kGroups;
  const size_t row = static_cast<size_t>(row0 + t);
  const int Hk = p.cache.Hk, heads = p.Hq + 2 * Hk;
  const int step = kGroups * static_cast<int>(gridDim.y);
  const int first = static_cast<int>(blockIdx.y) * kGroups + group % kGroups;
  const int rounds = (heads + step - 1) / step;
  const __nv_bfloat16* const y = p.y + row * heads * kD + 8 * c;
  const bool there = row0 + t < p.batch.rows;
  Chunk8 x[kWriteBatch];
  const auto load = [&](int r) {
#pragma unroll
    for (int b = 0; b < kWriteBatch; ++b) {
      const int h = first + (r + b) * step;
      x[b] = Chunk8{{0u, 0u, 0u, 0u}};
      if (there && h < heads && head_ok(p.batch, row, h, heads, kChkLoad)) x[b] = ldg8(y + h * kD);
    }
  };
  load(0);
  for (int i = warp; i < kTokens; i += kCacheThreads / 32) {
    const RowPlace pl = place_of(p.batch, p.cache, row0 + i, lane);
    if (lane == 0) place[i] = pl;
  }
  __syncthreads();
  for (int i = tid; i < kTokens * rope.half; i += kCacheThreads) {
    const int t = i / rope.half, j = i % rope.half;
    if (place[t].seq < 0) continue;
    const int64_t pos = rope.pos == nullptr
                            ? place[t].pos
                            : __ldg(rope.pos + static_cast<size_t>(rope.axis[j]) * p.batch.rows + row0 + t);
    const uint64_t phase = static_cast<uint64_t>(pos) * rope.turn[j];
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &sn[t][j], &cs[t][j]);
  }
  __syncthreads();

  const RowPlace pl = place[t];
  // (no thread leaves before the last shuffle: a warp's groups may be of different tokens)
  const int hc = rope.half / 8;  // 16-byte groups in half of the turned part
  const bool turned = c < 2 * hc;
  const bool pairs = rope.pairs != 0;
  const int i0 = pairs ? 4 * c : 8 * (c < hc ? c : c - hc);  // its first pair
  float cv[8], sv[8];  // of the pairs that its values are in
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = i0 + (pairs ? e / 2 : e);
    cv[e] = turned ? cs[t][i] : 1.0f;
    sv[e] = turned ? sn[t][i] : 0.0f;
    // the partner's sign: a' = a cos - b sin, b' = b cos + a sin
    if (pairs ? !(e & 1) : c < hc) sv[e] = -sv[e];
  }
  const int base = lane / kLanes * kLanes;  // the group's first lane in the warp
  const int partner = base + (pairs || !turned ? c : c < hc ? c + hc : c - hc);
#pragma unroll 1
  for (int r0 = 0; r0 < rounds; r0 += kWriteBatch) {
    if (r0 > 0) load(r0);
#pragma unroll
    for (int rb = 0; rb < kWriteBatch; ++rb) {
      const int h = first + (r0 + rb) * step;
      const bool in = pl.seq >= 0 && h < heads;
      const Chunk8 xv = x[rb];
      Chunk8 o = xv;
      if (!pairs) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o.w[e] = __shfl_sync(0xffffffffu, xv.w[e], partner);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o.w[e] = __byte_perm(xv.w[e], 0u, 0x1032);  // halves exchanged
      }
      float u[1][8], w[8];
      unpack8(xv, u[0]);
      unpack8(o, w);
      const bool is_v = h >= p.Hq + Hk;
      if (turned && !is_v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[0][e] = fmaf(w[e], sv[e], u[0][e] * cv[e]);
      }
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) amax = max3_abs_nan(amax, u[0][e], u[0][e + 1]);
#pragma unroll
      for (int o2 = kLanes / 2; o2 > 0; o2 >>= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o2));
      if (!in) continue;
      if (h < p.Hq) {
        if (!head_ok(p.batch, row, h, p.Hq, kChkStore)) continue;
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pack_bf16x2(u[0][2 * e], u[0][2 * e + 1]);
        stg8(p.q_out + (row * p.Hq + h) * kD + 8 * c, v);
      } else if (pl.page >= 0) {
        const size_t e = cache_entry(p.cache, pl.page, is_v ? h - p.Hq - Hk : h - p.Hq, pl.slot);
        if (!entries_ok(p.cache, e, 1)) continue;
        const Q8Factors f(amax);
        f.prepare(u);
        // (a key that is not turned is a bf16 number: the quantiser's rounding, whose first step, to 2^-15, takes 2^-16 of a
        // code from a turned one at most, a twentieth of what the turn's own rounding does)
        q8_store8<true>((is_v ? p.cache.v_q : p.cache.k_q) + e * kD + 8 * c, u[0], f);
        if (c == 0) (is_v ? p.cache.v_s : p.cache.k_s)[e] = q8_scale(amax);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Read: bf16(code * scale) of the rows' tokens, [rows, Hk, D] each of k and v.  Rows before their
// sequence's first token are zeros; a page that does not exist gives NaN.
// Bound by HBM: D + 4 bytes in, 2 D out per value row.  D / 16 threads share a (token, head), 16 codes
// each.
// ---------------------------------------------------------------------------
struct CacheReadParams {
  CacheQ8 cache;
  BatchQ8 batch;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
};

constexpr int kReadTokens = 16;

template <int kD>
__global__ void __launch_bounds__(kCacheThreads) cache_read_q8_kernel(const CacheReadParams p) {
  constexpr int kLanes = kD / 16;
  constexpr int kGroups = kCacheThreads / kLanes;  // (token, head) at a time
  __shared__ RowPlace place[kReadTokens];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int row0 = static_cast<int>(blockIdx.x) * kReadTokens;
  for (int i = warp; i < kReadTokens; i += kCacheThreads / 32) {
    const RowPlace pl = place_of(p.batch, p.cache, row0 + i, lane);
    if (lane == 0) place[i] = pl;
  }
  __syncthreads();
  const int c = tid % kLanes, Hk = p.cache.Hk;
  const int units = kReadTokens * Hk;  // token-major: neighbours write neighbouring heads
  const int step = kGroups * static_cast<int>(gridDim.y);
  // two units at a time, their loads together
  for (int u0 = static_cast<int>(blockIdx.y) * kGroups + tid / kLanes; u0 < units; u0 += 2 * step) {
    uint4 q[2][2];
    float s[2][2];
    size_t out[2];
    bool in[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int u = u0 + b * step, t = u / Hk, h = u - t * Hk;
      const RowPlace pl = place[min(t, kReadTokens - 1)];
      in[b] = u < units && pl.seq >= 0;
      out[b] = (static_cast<size_t>(row0 + t) * Hk + h) * kD + 16 * c;
      in[b] = in[b] && head_ok(p.batch, static_cast<size_t>(row0 + t), h, Hk, kChkStore);
      const bool there = in[b] && pl.page >= 0;
      const size_t e = there ? cache_entry(p.cache, pl.page, h, pl.slot) : 0;
      const bool held = there && entries_ok(p.cache, e, 1);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        q[b][kv] = make_uint4(0u, 0u, 0u, 0u);
        s[b][kv] = pl.pos < 0 ? 0.f : __int_as_float(0x7fffffff);
        if (held) {
          q[b][kv] = __ldcs(reinterpret_cast<const uint4*>((kv ? p.cache.v_q : p.cache.k_q) + e * kD + 16 * c));
          s[b][kv] = __ldg((kv ? p.cache.v_s : p.cache.k_s) + e);
        }
      }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if (!in[b]) continue;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t w[4] = {q[b][kv].x, q[b][kv].y, q[b][kv].z, q[b][kv].w};
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[4];
          q8_unpack4(w[i], f);
          v[2 * i] = pack_bf16x2(f[0] * s[b][kv], f[1] * s[b][kv]);
          v[2 * i + 1] = pack_bf16x2(f[2] * s[b][kv], f[3] * s[b][kv]);
        }
        __nv_bfloat16* o = (kv ? p.v_out : p.k_out) + out[b];
        __stcs(reinterpret_cast<uint4*>(o), make_uint4(v[0], v[1], v[2], v[3]));
        __stcs(reinterpret_cast<uint4*>(o + 8), make_uint4(v[4], v[5], v[6], v[7]));
      }
    }
  }
}

}  // namespace coda
