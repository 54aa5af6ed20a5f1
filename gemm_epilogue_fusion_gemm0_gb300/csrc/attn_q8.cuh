// attn_q8.cuh -- attention of new tokens over the 8-bit paged cache: the deal of the work, the kernel
// for few rows (decoding), and the join of parts.
//
//   o[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),  j <= lens - n + i
//   lse[i] = m_i + log sum_j p_ij
// i being one of a sequence's n new tokens, k_j and v_j the values of the cache's codes.  A row
// that sees no key is zero, its lse -inf.
//
// The rows of a sequence that share a key head, n tokens of `group` query heads each, are packed
// (row r is token r / group, head r % group) and cut into tiles; a tile with its keys is an item, and
// 128, 256 or 384 keys of it a unit.  Lengths are known to the device alone, so each block of a persistent grid
// adds up the units of all sequences, takes an equal, contiguous share of them, and walks it: whatever
// the lengths, all SMs end together, and a long sequence's keys are spread over as many blocks as its
// share of the work.  A part of an item leaves its running maximum, sum and unnormalised
// outputs in the workspace; a second kernel joins the parts of each such item in the order of its keys, so
// the same call gives the same bits every time.
#pragma once

#include <type_traits>

#include "cache_q8.cuh"

namespace coda {

constexpr int kAttnUnit = 128;       // keys of the kernel for tiles
constexpr int kFewKeys = 16;         // that a warp of the kernel for few takes together: a page holds them
constexpr int kFewStages = 2;
constexpr int kTileRows = 256, kTileThreads = 704;

// What the deal knows of a kernel.  kLead: measured, 64 sequences' decoding and chunks of 500 tokens.
// kN: groups of 8 rows (1 or 2); two have registers for 8 warps.
template <int kN>
struct FewDeal {
  static constexpr int kRows = 8 * kN, kWarps = kN == 1 ? 12 : 8, kThreads = 32 * kWarps, kLead = 1;
  static constexpr int kApart = kFewKeys * kWarps;  // from a warp's first 16 keys of a unit to its second
  static constexpr int kUnit = 2 * kApart;
};
struct TileDeal {
  static constexpr int kRows = kTileRows, kUnit = kAttnUnit, kThreads = kTileThreads, kLead = 3;
};
constexpr int kAttnMaxBlocks = 160;  // of the persistent grids

struct AttnQ8Params {
  const __nv_bfloat16* q;  // [rows, Hq, D]
  __nv_bfloat16* o;        // [rows, Hq, D]
  float* lse;              // [rows, Hq] or null
  CacheQ8 cache;
  BatchQ8 batch;
  int Hq, group;           // query heads; of them per key head
  // scale * log2 e, the part that is no power of two and the power.  The part goes into k's scales; what a row's products are
  // multiplied by in the exponents is then a power of two, so that a score less the largest is exact however large both are
  // (where the largest was a rounded product and the others were not, weights passed 2^15 with scores from 2^27 on, and
  // fp16's largest).
  float scale_part, scale_power;
};

// ---------------------------------------------------------------------------
// The deal
// ---------------------------------------------------------------------------
// A sequence as the call describes it, whatever cu and lens hold.
struct AttnSeq {
  int row0;   // its first row
  int n;      // rows of q that it has (0: none that exist)
  int first;  // token number of its first row; row i of it sees the keys 0 .. first + i
};

__host__ __device__ inline AttnSeq attn_seq(int cu0, int cu1, int len, int rows) {
  AttnSeq s;
  s.row0 = cu0;
  const int64_t n = static_cast<int64_t>(cu1 < rows ? cu1 : rows) - cu0;
  s.n = cu0 < 0 || n < 0 ? 0 : static_cast<int>(n);
  s.first = static_cast<int>(static_cast<int64_t>(len > 0 ? len : 0) - (static_cast<int64_t>(cu1) - cu0));
  return s;
}

// Keys that a tile of `tile_rows` packed rows sees at most.  `places`: tokens that the table has room
// for; a row that sees more is NaN by the first of them that has none, so none after it is walked.
// (Packed rows and tiles are 32-bit numbers: rows times heads of a call are.)
__host__ __device__ inline int attn_extent(const AttnSeq& s, int group, int tile_rows, int tile, int places) {
  const int all = s.n * group, room = all - tile * tile_rows;  // (tile * tile_rows < all)
  const int last = tile * tile_rows + (room < tile_rows ? room : tile_rows) - 1;
  const int64_t keys = static_cast<int64_t>(s.first) + last / group + 1;
  return keys <= 0 ? 0 : static_cast<int>(keys < places + 1 ? keys : places + 1);
}

// An item counts its units and kLead more, for what it costs to begin and to end one.
template <class K>
__host__ __device__ inline int attn_cost(int extent) {
  return K::kLead + (extent <= K::kUnit ? 1 : (extent + K::kUnit - 1) / K::kUnit);  // (an empty item still writes zeros)
}

__host__ __device__ inline int attn_tiles(const AttnSeq& s, int group, int tile_rows) {
  return static_cast<int>((static_cast<int64_t>(s.n) * group + tile_rows - 1) / tile_rows);
}

// Which sequences a launch takes: those of lo + 1 .. hi packed rows.
struct AttnDeal {
  int lo, hi;
};

__host__ __device__ inline bool attn_takes(const AttnDeal& d, const AttnSeq& s, int group) {
  return s.n * group > d.lo && s.n * group <= d.hi;
}

// Where block c's share of the launch's cost begins.
__host__ __device__ inline int64_t attn_share(int64_t cost, int c, int blocks) {
  return cost * c / blocks;
}

// An item that begins in block c's share and does not end there: what the join needs to know.
struct AttnCut {
  int64_t cost;     // of the launch
  int64_t end;      // where the item ends in it
  int b, hk, tile;
  int valid;
};

// Of the kernel for few, with the sequence itself: one load less to wait for in the join (one token over 131072 keys
// 59.6 -> 57.1 us; among tiles the longer record costs more than it gives, a prompt of 8192 572 -> 580).
struct AttnCutFew {
  AttnCut cut;
  AttnSeq s;
  int pad;
};


struct AttnWs {
  AttnCutFew* cut;  // [blocks]; of tiles `cut` alone
  float2* ml;       // [2 blocks][rows]: what was taken out of the exponents (base 2), and the sum
  float* unit;      // [2 blocks][rows]: what the outputs are to be multiplied by
  float* o;         // [2 blocks][rows][D]
  int tile;         // rows of a tile
  int rows;         // of a part: as many as the call's tiles may have
};

__device__ __forceinline__ AttnSeq load_seq(const AttnQ8Params& p, int b) {
  return attn_seq(__ldg(p.batch.cu + b), __ldg(p.batch.cu + b + 1), __ldg(p.batch.lens + b), p.batch.rows);
}

// Where a block is in its share.
struct AttnWalk {
  AttnSeq s;
  int b, hk;
  int tile, tiles;
  int extent, cost;  // of the item
  int at;            // how much of its cost has been taken, by this block and those before it
  int unit, last;    // units of the piece in hand: unit .. last - 1
  bool begins, ends;  // the piece has the item's first unit; its last
  int64_t left;      // of the share
};

template <class K>
__device__ __forceinline__ void walk_item(AttnWalk& w, const AttnQ8Params& p, int places) {
  w.extent = attn_extent(w.s, p.group, K::kRows, w.tile, places);
  w.cost = attn_cost<K>(w.extent);
}

// The next piece: the units of one item that lie in the share.  False at the share's end.  (A share that ends or
// begins in what an item counts beyond its units has none of them, or all.)
template <class K>
__device__ __forceinline__ bool walk_piece(AttnWalk& w, const AttnQ8Params& p, const AttnDeal& d, int places) {
  while (w.left > 0) {
    if (w.at == w.cost) {
      w.at = 0;
      if (++w.tile == w.tiles) {
        w.tile = 0;
        if (++w.hk == p.cache.Hk) {
          w.hk = 0;
          do {
            ++w.b;
            if (w.b >= p.batch.B) return false;  // (cu or lens written while the call runs)
            w.s = load_seq(p, w.b);
          } while (!attn_takes(d, w.s, p.group));
          w.tiles = attn_tiles(w.s, p.group, K::kRows);
        }
      }
      walk_item<K>(w, p, places);
    }
    const int rest = w.cost - w.at, n = w.left < rest ? static_cast<int>(w.left) : rest;
    w.unit = max(w.at - K::kLead, 0);
    w.last = max(w.at + n - K::kLead, 0);
    w.at += n;
    w.left -= n;
    w.begins = w.unit == 0;
    w.ends = n == rest;
    if (w.unit < w.last) return true;
  }
  return false;
}

// The next unit, in this piece or in the next.
template <class K>
__device__ __forceinline__ bool walk_unit(AttnWalk& w, const AttnQ8Params& p, const AttnDeal& d, int places) {
  return ++w.unit < w.last || walk_piece<K>(w, p, d, places);
}

// Cost of a sequence for one key head, by a whole warp (0: another launch's sequence).
template <class K>
__device__ __forceinline__ int64_t seq_cost(const AttnSeq& s, const AttnQ8Params& p, const AttnDeal& d, int places,
                                            int lane) {
  if (!attn_takes(d, s, p.group)) return 0;
  const int tiles = attn_tiles(s, p.group, K::kRows);
  int64_t u = 0;
  for (int t = lane; t < tiles; t += 32) u += attn_cost<K>(attn_extent(s, p.group, K::kRows, t, places));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u;
}

// Adds up the costs (all threads of the block), and puts the walk at the beginning of this block's share, before
// its first piece.  Returns the launch's cost; `end`: where the share ends in it.  False in `some`: an empty share.  A
// warp adds up a sequence at a time, a lane a tile; `costs` (shared memory, at least B numbers) holds the
// sequences' sums in between.
template <class K>
__device__ __forceinline__ int64_t walk_start(AttnWalk& w, const AttnQ8Params& p, const AttnDeal& d, int places,
                                              int64_t* costs, int64_t& end, bool& some) {
  constexpr int kThreads = K::kThreads;
  __shared__ int64_t warp_sum[kThreads / 32];
  __shared__ int64_t start_rest;
  __shared__ int start_b;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  for (int b = warp; b < p.batch.B; b += kThreads / 32) {
    const int64_t u = seq_cost<K>(load_seq(p, b), p, d, places, lane);
    if (lane == 0) costs[b] = u;
  }
  __syncthreads();
  const int per = (p.batch.B + kThreads - 1) / kThreads;
  const int b0 = min(p.batch.B, tid * per), b1 = min(p.batch.B, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += costs[b] * p.cache.Hk;
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) upto += warp_sum[i];
    total += warp_sum[i];
  }
  const int64_t begin = attn_share(total, blockIdx.x, gridDim.x);
  end = attn_share(total, blockIdx.x + 1, gridDim.x);
  some = begin < end;
  if (some && upto - mine <= begin && begin < upto) {  // one thread: the share begins in its sequences
    int64_t rest = begin - (upto - mine);
    int b = b0;
    for (; rest >= costs[b] * p.cache.Hk; ++b) rest -= costs[b] * p.cache.Hk;
    start_b = b;
    start_rest = rest;
  }
  __syncthreads();
  if (!some) return total;
  w.b = start_b;
  w.s = load_seq(p, w.b);
  w.tiles = attn_tiles(w.s, p.group, K::kRows);
  int64_t rest = start_rest;
  const int64_t per_head = costs[w.b];
  w.hk = static_cast<int>(rest / per_head);
  rest -= w.hk * per_head;
  for (w.tile = 0;; w.tile += 32) {  // 32 tiles at a time
    const int t = w.tile + lane;
    const int u = t < w.tiles ? attn_cost<K>(attn_extent(w.s, p.group, K::kRows, t, places)) : 0;
    int64_t before = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += v;
    }
    const uint32_t here = __ballot_sync(0xffffffffu, rest < before);
    if (here != 0u || w.tile + 32 >= w.tiles) {
      const int at = here != 0u ? __ffs(here) - 1 : 31;
      rest -= __shfl_sync(0xffffffffu, before - u, at);
      w.tile += at;
      break;
    }
    rest -= __shfl_sync(0xffffffffu, before, 31);
  }
  walk_item<K>(w, p, places);
  w.at = static_cast<int>(rest);
  w.left = end - begin;
  __syncthreads();  // `costs` is read: its memory is free
  return total;
}

// Tells the join of the item whose piece `w` is, if it begins here and ends elsewhere.
__device__ __forceinline__ void tell_cut(const AttnWalk& w, AttnCut* cut, int64_t total, int64_t end) {
  if (w.begins && !w.ends) *cut = AttnCut{total, end - w.left + (w.cost - w.at), w.b, w.hk, w.tile, 1};
}

// Row `packed` of a sequence's rows that share a key head: its row of q and its query head.
struct AttnRow {
  int64_t at;  // row * Hq + head
  int limit;   // the last key that it sees
  bool in;     // false behind the sequence's last (`at` and `limit` are then the last's)
};

__device__ __forceinline__ AttnRow attn_row(const AttnQ8Params& p, const AttnSeq& s, int hk, int packed) {
  AttnRow r;
  const int all = s.n * p.group;
  r.in = packed < all;
  const int i = (r.in ? packed : all - 1) / p.group;
  r.limit = s.first + i;
  r.at = static_cast<int64_t>(s.row0 + i) * p.Hq + hk * p.group + ((r.in ? packed : all - 1) - i * p.group);
  return r;
}

// That row's head lies within q and o (in the checked build).
__device__ __forceinline__ bool row_ok(const AttnQ8Params& p, const AttnRow& r, uint32_t site) {
  return checked(r.at >= 0 && r.at < static_cast<int64_t>(p.batch.rows) * p.Hq, site);
}
// Row `row` of a block's part `slot` lies within the workspace (the same).
__device__ __forceinline__ bool part_ok(const AttnWs& ws, size_t slot, int row) {
  return checked(slot < size_t(2) * kAttnMaxBlocks && row >= 0 && row < ws.rows, kChkPart);
}

// Natural logarithm of a row's sum (0: it sees no key) with the maximum `top` taken out, in base 2.
__device__ __forceinline__ float attn_lse(float top, float sum) {
  return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

// ---------------------------------------------------------------------------
// Few rows: tiles of 8 or 16
//
// Bound by HBM: 2 (D + 4) bytes per key, used for at most 16 rows.  As in the product for few tokens, each
// warp has its own ring: 2 x 16 keys of a unit (so that a short context is spread over all warps too), codes and
// scales, by cp.async up to two units ahead, and no barrier but the warp's in the loop.  The pages of a unit are looked
// up one unit before its copies start.  Its instructions are the nearer bound, most of them the widening of codes,
// so the keys are the 16 rows of an instruction and the query rows its 8 columns:
//   S^T = k q^T,  o^T += v^T p^T    mma.sync.m16n8k16 on fp16
// which takes half the instructions of the products and of the softmax that 16 query rows to an instruction take where
// there are at most 8 (one token of 8 heads to a key head), and registers for 12 warps in place of 8: 64 tokens over up
// to 8192 keys each, 64 / 8 heads of 128, 127 us, 5.4 TB/s (rows as the instruction's rows, before the powers below: 144,
// with these 124).
//
// q's rows are brought into fp16's range by a power of two each (exact); codes are exact in fp16 (1024 + 128 + code by
// bits, less 1152).  A thread (g = lane / 4, t = lane % 4) reads 16 codes of keys g and g + 8 at a time: its operand k
// of 2 t, 2 t + 1, 2 t + 8, 2 t + 9 are four neighbouring values, the same of q.  It has the scores of these keys and of
// rows 2 t, 2 t + 1; their weights change places by movmatrix to keys 2 t, 2 t + 1 of row g.  For v^T p^T it reads 16
// values (8 for D = 64) of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9, rows g and g + 8 of tile j being values 2 j and 2 j + 1 of
// the g-th 16.  Both reads are free of bank conflicts with the 16-byte groups of a key exchanged as below.
//
// Scales: a key's multiplies its row of S^T; a value's, less a power of two, its row of p^T.  What is taken out of the
// exponents is a row's largest score, rounded up to a whole number, so that a weight's rounding to fp16 is the same whatever
// keys a part began with (else 11 % of the outputs changed with the rest of the batch); it moves, and sum and outputs
// with it, only where p would pass 2^8, which a thread sees in its own scores; only then is a row's maximum found.  The
// power of two is the largest value scale's, rounded up, so that weights times scales stay within fp16; a row's own, of the
// keys that it sees, where a unit has keys that some rows do not see.  It is the outputs' alone: a sum that shared it
// (weights of 2^(score - maximum - power)) lost its small terms, then all, with scales from 2^102 on.
//
// The product with v's codes, which are exact in fp16, takes weights times scales in fp16 too: 2^-11 of each at most, an
// eighth of what the outputs' rounding to bf16 may take.  (A second product for what is rounded away would cost as much as
// the first.)  The sum of weights is of the numbers before that.
// ---------------------------------------------------------------------------
template <int kD, int kN>
struct FewSmem {
  static constexpr int kWarps = FewDeal<kN>::kWarps;
  static constexpr int kMeet = kN == 1 ? 4 : 16;  // rows whose parts meet at a time: what there is room for
  static constexpr uint32_t kCodes = kFewKeys * kD;                  // of 16 keys
  static constexpr uint32_t kGroup = 2 * kCodes + 2 * kFewKeys * 4;  // k, v, their scales
  static constexpr uint32_t kStage = 2 * kGroup;
  static constexpr uint32_t kJoin = kWarps * kFewStages * kStage;    // the warps' outputs
  static constexpr uint32_t kEnd = kJoin + kWarps * kMeet * kD * 4;
  static constexpr uint32_t kBytes = kEnd > 65536 ? kEnd : 65536;    // (the sequences' costs at the start)
  static_assert(kGroup % 128 == 0 && kBytes <= 232448u - 4096u, "shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The power of two that brings a row with the given largest magnitude to 2^14 .. 2^15 in fp16 (as
// near as fp32 has one), and its reciprocal.  A NaN or an infinity gives a reciprocal of NaN.
__device__ __forceinline__ void row_power(float amax, float& up, float& down) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  const int f = min(14 - e, 126);
  up = __uint_as_float(static_cast<uint32_t>(f + 127) << 23);
  down = f < 0 || f <= 126 ? __uint_as_float(static_cast<uint32_t>(127 - f) << 23) : 0.f;
  if (!(amax <= 3.402823466e38f)) {
    up = 0.f;
    down = __int_as_float(0x7fffffff);
  }
}

// What a row's products are multiplied by in the exponents; never zero, which times a masked score's -inf is NaN.
__device__ __forceinline__ float exponent_factor(float scale_power, float down) {
  const float f = scale_power * down;
  return f < 1.17549435e-38f ? 1.17549435e-38f : f;
}

// The power of two that a value scale is at most (2^-60 for smaller ones, a NaN among them; an infinity stands for 2^128).
constexpr float kLeastScale = 0x1p-60f;
__device__ __forceinline__ float finite_size(float s) { return fabsf(s) <= 3.402823466e38f ? fabsf(s) : 0.f; }
__device__ __forceinline__ float scale_power(float s) {
  return s > kLeastScale ? __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u) : kLeastScale;
}
// A value scale goes into the weights divided by power / 2^kPowerUp, and the outputs are multiplied by that in the end
// (both are fp32 numbers for all powers).  A weight is at most 2^8, so the products reach 2^15 at most (fp16 has 65504), and
// a row's largest weights begin at 2^5 or above: those down to 2^-20 of them keep fp16's 11 bits.  (With products from one
// down, 131072 alike of 2^-17 beside a large one were 5e-3 off, all to one side.)
constexpr uint32_t kPowerUp = 7;
__device__ __forceinline__ float power_unit(float power) {
  return __uint_as_float(__float_as_uint(power) - (kPowerUp << 23));
}
__device__ __forceinline__ float power_inverse(float power) {
  return __uint_as_float(((254u + kPowerUp) << 23) - __float_as_uint(power));
}
// a / b of powers of two at most 2^126 apart; and the power half way between two, which is that near to any between them.
__device__ __forceinline__ float power_ratio(float a, float b) {
  return __uint_as_float(__float_as_uint(a) - __float_as_uint(b) + (127u << 23));
}
__device__ __forceinline__ float power_between(float a, float b) {
  return __uint_as_float((__float_as_uint(a) / 2 + __float_as_uint(b) / 2) & 0x7f800000u);
}
// log2 of a / b, powers of two
__device__ __forceinline__ float power_log2(float a, float b) {
  return static_cast<float>(static_cast<int>(__float_as_uint(a) >> 23) - static_cast<int>(__float_as_uint(b) >> 23));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// max(|a|, |b|, |c|), of those that are numbers
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Four codes of a word to fp16, in order
__device__ __forceinline__ void q8_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = q8_less_1152(__byte_perm(u, 0x64646464u, 0x4140));
  hi = q8_less_1152(__byte_perm(u, 0x64646464u, 0x4342));
}

// Where the 16-byte group c of key r of a stage sits, for k and for v (8 groups of 16 bytes are a line
// of 128; a key is one line, or half of one).  Eight lanes read together: keys g = 0, 1 with groups
// t = 0..3 of k; keys 0, 2, 4, 6 with groups 0, 1 (halves of them: D = 64) of v.
template <int kD>
__device__ __forceinline__ uint32_t few_k_at(uint32_t r, uint32_t c) {
  if constexpr (kD == 128) return 128u * r + 16u * (c ^ ((r & 1u) << 2));
  return 128u * (r >> 1) + 16u * (((r & 1u) << 2 | c) ^ ((r >> 1 & 3u) << 1));
}
template <int kD>
__device__ __forceinline__ uint32_t few_v_at(uint32_t r, uint32_t c) {
  if constexpr (kD == 128) return 128u * r + 16u * (c ^ (r & 6u));
  return 128u * (r >> 1) + 16u * (((r & 1u) << 2 | c) ^ ((r >> 1 & 3u) << 1));
}

// An 8 x 8 matrix of 16-bit numbers, two columns 2 t, 2 t + 1 of row g in a register, to its transpose.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The power of the largest scale that a row sees of a warp's 32 keys: s0 .. s3 are those of this thread's first key and of
// those 8, apart and apart + 8 behind it, of which the row sees 0 .. seen.  (Not inlined: hardly ever called.)
__device__ __noinline__ float seen_power(float s0, float s1, float s2, float s3, int seen, int apart) {
  float top = 0 <= seen ? finite_size(s0) : 0.f;
  if (8 <= seen) top = fmaxf(top, finite_size(s1));
  if (apart <= seen) top = fmaxf(top, finite_size(s2));
  if (apart + 8 <= seen) top = fmaxf(top, finite_size(s3));
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  return scale_power(top);
}

template <int kD, int kN>
__global__ void __launch_bounds__(FewDeal<kN>::kThreads, 1)
    attn_q8_few_kernel(const AttnQ8Params p, const AttnWs ws, const AttnDeal deal) {
  using Smem = FewSmem<kD, kN>;
  using Deal = FewDeal<kN>;
  constexpr int kSteps = kD / 16;   // instructions along D of S^T
  constexpr int kTiles = kD / 16;   // tiles of 16 rows of o^T
  constexpr int kF4 = kD / 32;      // float4s of a row of o in a thread
  constexpr int kWarps = Deal::kWarps, kMeet = Smem::kMeet;
  extern __shared__ __align__(1024) uint8_t smem_few[];
  __shared__ float2 warp_ml[kWarps][8 * kN];
  __shared__ float2 row_ml[8 * kN];
  const int lane = threadIdx.x & 31;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int g = lane >> 2, t = lane & 3;
  const int places = p.batch.width << p.cache.page_log2;
  const uint32_t ring = smem_u32(smem_few) + static_cast<uint32_t>(warp) * kFewStages * Smem::kStage;
  float4* const join = reinterpret_cast<float4*>(smem_few + Smem::kJoin);
  griddep_launch_dependents();
  griddep_wait();

  AttnWalk w;
  int64_t end;
  bool some;
  const int64_t total = walk_start<Deal>(w, p, deal, places, reinterpret_cast<int64_t*>(smem_few), end, some);
  if (threadIdx.x == 0) ws.cut[blockIdx.x].cut.valid = 0;
  if (!some || !walk_piece<Deal>(w, p, deal, places)) return;
  const int mine = warp * kFewKeys;  // the warp's first key of a unit
  const int mask = (1 << p.cache.page_log2) - 1;
  AttnWalk ahead = w;
  // the table's entry for the warp's first (even lanes) and second 16 keys of a unit
  const auto entry_at = [&](const AttnWalk& a) {
    const int key = a.unit * Deal::kUnit + mine + Deal::kApart * (lane & 1), i = key >> p.cache.page_log2;
    return key < a.extent && i < p.batch.width ? __ldg(p.batch.table + static_cast<size_t>(a.b) * p.batch.width + i) : -1;
  };
  int entry = entry_at(ahead);
  uint32_t issued = 0;
  bool more = true;  // units to ask for
  constexpr int kChunks = kD / 16;
  // this thread's 16 codes of a copy: key kr (+ 32 / kChunks for the next), group kc
  const uint32_t kr = lane / kChunks, kc = lane % kChunks;
  const uint32_t lane_at = kr * kD + 16 * kc;
  const auto issue = [&]() {  // the unit `ahead` is at
    const uint32_t st = ring + (issued & (kFewStages - 1)) * Smem::kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = ahead.unit * Deal::kUnit + mine + Deal::kApart * h;
      const int page = __shfl_sync(0xffffffffu, entry, h);
      if (key >= ahead.extent) continue;
      const uint32_t gr = st + h * Smem::kGroup;
      const uint32_t sc = gr + 2 * Smem::kCodes + 4u * lane;  // k's 16 scales, then v's
      if (static_cast<unsigned>(page) < static_cast<unsigned>(p.cache.pages)) {
        const size_t e = cache_entry(p.cache, page, ahead.hk, key & mask);
        if (!entries_ok(p.cache, e, kFewKeys)) continue;
        const uint8_t* const k = p.cache.k_q + e * kD + lane_at;
        const uint8_t* const v = p.cache.v_q + e * kD + lane_at;
#pragma unroll
        for (int i = 0; i < kFewKeys * kChunks / 32; ++i) {
          const uint32_t r = i * (32 / kChunks) + kr;
          cp_async16(gr + few_k_at<kD>(r, kc), k + i * 512);
          cp_async16(gr + Smem::kCodes + few_v_at<kD>(r, kc), v + i * 512);
        }
        cp_async4(sc, (lane < 16 ? p.cache.k_s : p.cache.v_s) + e + (lane & 15));
      } else {
        if (lane == 0) atomicCAS(&g_coda_status, 0u, 0x200u | kChkPage);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sc), "r"(0x7fffffff) : "memory");
      }
    }
    ++issued;
    more = walk_unit<Deal>(ahead, p, deal, places);
    if (more) entry = entry_at(ahead);
  };
#pragma unroll
  for (int i = 0; i < kFewStages; ++i) {
    if (more) issue();
    cp_async_commit();
  }

  uint32_t used = 0;
  do {
    // a piece of an item: its rows of q, row 8 n + g in this thread; then of rows 8 n + 2 t + e their factor and limit
    uint32_t qb[kN][kSteps][2];
    float acc[kN][kTiles][4];
    float l[kN][2], rf[kN][2], base[kN][2];
    float power[kN][2];  // of the value scales, in the outputs
    // what the value scales are divided by: the power where all of the warp's rows have one (`fit` too; else it is negative)
    float common = kLeastScale, fit = kLeastScale;
    int limit[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const AttnRow row = attn_row(p, w.s, w.hk, w.tile * Deal::kRows + 8 * n + g);
      Chunk8 c[kSteps / 2];
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        c[i] = Chunk8{{0u, 0u, 0u, 0u}};
        if (row.in && row_ok(p, row, kChkLoad)) c[i] = ldg8(p.q + row.at * kD + 64 * (i / 2) + 16 * t + 8 * (i % 2));
      }
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        float v[8];
        unpack8(c[i], v);
#pragma unroll
        for (int e = 0; e < 8; e += 2) amax = max3_abs_nan(amax, v[e], v[e + 1]);
      }
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up, down;
      row_power(amax, up, down);
      // (a row that sees no token is zero whatever it holds: its scores, all -inf, times a NaN would not be)
      const float factor = row.limit < 0 ? 1.0f : exponent_factor(p.scale_power, down);
#pragma unroll
      for (int i = 0; i < kSteps / 2; ++i) {
        float v[8];
        unpack8(c[i], v);
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // two instructions of four values each
          const float* x = v + 4 * e;
          qb[n][2 * i + e][0] = pack_f16x2(x[0] * up, x[1] * up);
          qb[n][2 * i + e][1] = pack_f16x2(x[2] * up, x[3] * up);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        rf[n][e] = __shfl_sync(0xffffffffu, factor, 4 * (2 * t + e));
        limit[n][e] = __shfl_sync(0xffffffffu, row.limit, 4 * (2 * t + e));
        base[n][e] = -INFINITY;
        l[n][e] = 0.f;
        power[n][e] = kLeastScale;
      }
#pragma unroll
      for (int j = 0; j < kTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.f;
    }
    const int low = w.s.first + w.tile * Deal::kRows / p.group;  // the smallest limit
    for (; w.unit < w.last; ++w.unit, ++used) {
      cp_async_wait<kFewStages - 1>();
      __syncwarp();
      const int key = w.unit * Deal::kUnit + mine;
      if (key < w.extent) {
        const bool two = key + Deal::kApart < w.extent;  // the second 16 too
        const uint32_t st = ring + (used & (kFewStages - 1)) * Smem::kStage;
        // scores of keys g (e < 2) and g + 8 of the first 16 and of the second, rows 8 n + 2 t + e % 2
        float s[2][kN][4] = {};
        float ks[2][2], vs[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1 && !two) continue;
          const uint32_t gr = st + q * Smem::kGroup;
#pragma unroll
          for (int h = 0; h < kD / 64; ++h) {
            const uint4 c0 = ld_shared_v4(gr + few_k_at<kD>(g, 4 * h + t));
            const uint4 c1 = ld_shared_v4(gr + few_k_at<kD>(g + 8, 4 * h + t));
            const uint32_t x[4] = {c0.x, c0.y, c0.z, c0.w}, y[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a0, a1, a2, a3;
              q8_to_f16x2(x[i], a0, a2);
              q8_to_f16x2(y[i], a1, a3);
#pragma unroll
              for (int n = 0; n < kN; ++n)
                mma_f16_16816(s[q][n], a0, a1, a2, a3, qb[n][4 * h + i][0], qb[n][4 * h + i][1]);
            }
          }
          const float* const sc =
              reinterpret_cast<const float*>(smem_few + (gr - smem_u32(smem_few)) + 2 * Smem::kCodes) + g;
          ks[q][0] = sc[0] * p.scale_part, ks[q][1] = sc[8] * p.scale_part;
          vs[q][0] = sc[16], vs[q][1] = sc[24];
        }
        if (!two) ks[1][0] = ks[1][1] = vs[1][0] = vs[1][1] = 0.f;
        const auto key_of = [&](int q, int e) { return key + Deal::kApart * q + g + 8 * e; };
        const bool edge = key + Deal::kApart + kFewKeys - 1 > low;
        if (edge) {  // what lies behind the last key is not looked at
          __syncwarp();  // (a branch, which predicates instead would cost every unit)
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key_of(q, e) >= w.extent) vs[q][e] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[q][n][e] *= ks[q][e >> 1];
        if (edge) {
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key_of(q, e >> 1) > limit[n][e & 1]) s[q][n][e] = -INFINITY;
        }
        float mx[kN][2];
        bool fits = fmaxf(max3_abs(0.f, vs[0][0], vs[0][1]), max3_abs(0.f, vs[1][0], vs[1][1])) <= fit;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[n][e] = max3(fmaxf(s[0][n][e], s[0][n][2 + e]), s[1][n][e], s[1][n][2 + e]);
            fits = fits && mx[n][e] * rf[n][e] <= base[n][e] + 8.0f;
          }
        if (!__all_sync(0xffffffffu, fits)) {
          float less[kN][2];  // what the outputs are multiplied by for the powers
          const auto most = [&](int limit) {
            return seen_power(vs[0][0], vs[0][1], vs[1][0], vs[1][1], max(limit, -1) - key - g, Deal::kApart);
          };
          const float all = fmaxf(common, most(0x7fffffff));
          if (!edge || all <= fit) {
            const float by = ex2(power_log2(common, all));
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) power[n][e] = all, less[n][e] = by;
            common = fit = all;
          } else {
            float high = 0.f, low_power = INFINITY;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float before = power[n][e];
                power[n][e] = fmaxf(before, most(limit[n][e]));
                less[n][e] = ex2(power_log2(before, power[n][e]));
                high = fmaxf(high, power[n][e]);
                low_power = fminf(low_power, power[n][e]);
              }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
              high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
              low_power = fminf(low_power, __shfl_xor_sync(0xffffffffu, low_power, o));
            }
            common = power_between(low_power, high);
            fit = low_power == high ? high : -1.0f;
          }
#pragma unroll
          for (int n = 0; n < kN; ++n) {
            float c[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int o = 4; o <= 16; o <<= 1)
                mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
              const float to_be = mx[n][e] * rf[n][e];
              c[e] = 1.0f;
              if (to_be > base[n][e] + 8.0f) {
                c[e] = ex2(base[n][e] - ceilf(to_be));
                base[n][e] = ceilf(to_be);
              }
              l[n][e] *= c[e];
              c[e] *= less[n][e];
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[n][j][e] *= c[e & 1];
          }
        }
        uint32_t pb[2][kN][2];  // weights of keys 2 t, 2 t + 1 (and 8 further) of row 8 n + g
        const float by = power_inverse(common);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) vs[q][e] *= by;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          const float less[2] = {base[n][0] == -INFINITY ? 0.f : base[n][0],  // (no key seen yet)
                                 base[n][1] == -INFINITY ? 0.f : base[n][1]};
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = ex2(fmaf(s[q][n][e], rf[n][e & 1], -less[e & 1]));
              l[n][e & 1] += x;
              s[q][n][e] = x * vs[q][e >> 1];
            }
        }
        if (edge) {  // (a scale behind a row's last key may be anything)
          __syncwarp();
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float own = power_ratio(common, power[n][e & 1]);
#pragma unroll
              for (int q = 0; q < 2; ++q) s[q][n][e] = key_of(q, e >> 1) > limit[n][e & 1] ? 0.f : s[q][n][e] * own;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              pb[q][n][e] = transposed(pack_f16x2(s[q][n][2 * e], s[q][n][2 * e + 1]));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 1 && !two) continue;
          uint32_t v[4][kD / 32];  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9: kD / 8 values of each
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t r = 8 * (i >> 1) + 2 * t + (i & 1);
            const uint32_t at = st + q * Smem::kGroup + Smem::kCodes;
            if constexpr (kD == 128) {
              const uint4 x = ld_shared_v4(at + few_v_at<kD>(r, g));
              v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
            } else {
              asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                           : "=r"(v[i][0]), "=r"(v[i][1])
                           : "r"(at + few_v_at<kD>(r, g >> 1) + 8u * (g & 1))
                           : "memory");
            }
          }
#pragma unroll
          for (int i = 0; i < kD / 32; ++i) {
            uint32_t b[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t x = v[2 * h][i] ^ 0x80808080u, y = v[2 * h + 1][i] ^ 0x80808080u;
              const uint32_t lo = __byte_perm(x, y, 0x5140), hi = __byte_perm(x, y, 0x7362);
              b[h][0] = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4140));
              b[h][1] = q8_less_1152(__byte_perm(lo, 0x64646464u, 0x4342));
              b[h][2] = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4140));
              b[h][3] = q8_less_1152(__byte_perm(hi, 0x64646464u, 0x4342));
            }
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              mma_f16_16816(acc[n][2 * i], b[0][0], b[0][1], b[1][0], b[1][1], pb[q][n][0], pb[q][n][1]);
              mma_f16_16816(acc[n][2 * i + 1], b[0][2], b[0][3], b[1][2], b[1][3], pb[q][n][0], pb[q][n][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage is read (and used: what was read is in registers)
      if (more) issue();
      cp_async_commit();
    }

    // The warps' parts meet.
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
        if (g == 0) warp_ml[warp][8 * n + 2 * t + e] = make_float2(base[n][e], l[n][e]);
      }
    __syncthreads();
    const int rows = min(Deal::kRows, w.s.n * p.group - w.tile * Deal::kRows);
    float f[kN][2];  // of the warp's parts
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) top = fmaxf(top, warp_ml[i][r].x);
        const float less = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 x = warp_ml[i][r];
          sum = fmaf(x.y, ex2(x.x - less), sum);
        }
        if (warp == 0 && g == 0) row_ml[r] = make_float2(top, sum);
        // (as quotients by the sum, within 2 ulp, which stay in range whatever the power)
        f[n][e] = ex2(base[n][e] - less) * (sum == 0.f ? 0.f : __fdividef(power_unit(power[n][e]), sum));
      }
    const bool whole = w.begins && w.ends;
    const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (w.begins ? 1 : 0);
#pragma unroll
    for (int q = 0; q < 8 * kN / kMeet; ++q) {  // rows kMeet q ..
      if (q * kMeet >= rows) continue;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * n + 2 * t + e - q * kMeet;
          if (r < 0 || r >= kMeet) continue;
#pragma unroll
          for (int i = 0; i < kF4; ++i) {
            const float(&a)[kTiles][4] = acc[n];
            const float by = f[n][e];
            join[(warp * kMeet + r) * (kD / 4) + kF4 * g + (i ^ (g & (kF4 - 1)))] = make_float4(
                a[2 * i][e] * by, a[2 * i][2 + e] * by, a[2 * i + 1][e] * by, a[2 * i + 1][2 + e] * by);
          }
        }
      __syncthreads();
      for (int i = threadIdx.x; i < min(kMeet, rows - q * kMeet) * (kD / 4); i += Deal::kThreads) {
        const int jr = i / (kD / 4), c = i % (kD / 4), row_at = q * kMeet + jr;
        const int at = c / kF4 * kF4 + ((c % kF4) ^ (c / kF4 & (kF4 - 1)));
        float4 x = join[jr * (kD / 4) + at];
#pragma unroll
        for (int k = 1; k < kWarps; ++k) {
          const float4 y = join[(k * kMeet + jr) * (kD / 4) + at];
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float2 ml = row_ml[row_at];
        if (whole) {
          const AttnRow row = attn_row(p, w.s, w.hk, w.tile * Deal::kRows + row_at);
          if (!row_ok(p, row, kChkStore)) continue;
          *reinterpret_cast<uint2*>(p.o + row.at * kD + 4 * c) =
              make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
          if (c == 0 && p.lse != nullptr) p.lse[row.at] = attn_lse(ml.x, ml.y);
        } else if (part_ok(ws, slot, row_at)) {
          reinterpret_cast<float4*>(ws.o)[(slot * ws.rows + row_at) * (kD / 4) + c] = x;
          if (c == 0) {
            ws.ml[slot * ws.rows + row_at] = ml;
            ws.unit[slot * ws.rows + row_at] = ml.y;
          }
        }
      }
      __syncthreads();  // the rows' place is free
    }
    if (threadIdx.x == 0) {
      ws.cut[blockIdx.x].s = w.s;
      tell_cut(w, &ws.cut[blockIdx.x].cut, total, end);
    }
  } while (walk_piece<Deal>(w, p, deal, places));
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// The join of an item's parts: block (c, y) has up to 16 rows of the item whose first part ends block c's share;
// the parts follow in the next blocks' first slots.  The parts' weights are formed once, then a thread adds
// four columns of a row over the parts, in order.  y = 0: of the launch for few; 1 ..: rows 16 (y - 1) ..
// of the launch for tiles; of both in one launch.
// ---------------------------------------------------------------------------
template <int kD>
__global__ void __launch_bounds__(256)
    attn_q8_join_kernel(const AttnQ8Params p, const AttnWs few, const AttnWs tiles, int y0, int blocks) {
  constexpr int kGroup = 16;
  __shared__ float weight[kAttnMaxBlocks][kGroup];
  __shared__ int slots[kAttnMaxBlocks];
  __shared__ float2 row_ml[kGroup];
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x, tid = static_cast<int>(threadIdx.x), y = static_cast<int>(blockIdx.y) + y0;
  const AttnWs& ws = y == 0 ? few : tiles;
  const int kRows = ws.tile, slot_rows = ws.rows;
  const AttnCut cut = ws.cut[c].cut;
  AttnSeq s;
  if (y == 0) s = ws.cut[c].s;
  if (!cut.valid) return;
  if (y != 0) s = load_seq(p, cut.b);
  const int r0 = y == 0 ? 0 : (y - 1) * kGroup;
  const int rows = min(min(kGroup, kRows - r0), s.n * p.group - cut.tile * kRows - r0);
  if (rows <= 0) return;
  // blocks c .. c + parts - 1; one whose share is empty (fewer units than blocks) has no part
  const int parts = static_cast<int>((cut.end * blocks + cut.cost - 1) / cut.cost) - c;
  for (int j = tid; j < parts; j += 256) {
    const bool has = attn_share(cut.cost, c + j, blocks) < attn_share(cut.cost, c + j + 1, blocks) &&
                     part_ok(ws, 2 * static_cast<size_t>(c + j) + 1, r0 + rows - 1);
    slots[j] = has ? 2 * (c + j) + (j == 0 ? 1 : 0) : -1;
  }
  __syncthreads();
  {  // a half warp per row
    const int r = tid >> 4, l = tid & 15;
    float top = -INFINITY, sum = 0.f;
    for (int j = l; j < parts; j += 16)
      if (slots[j] >= 0 && r < rows) {
        top = fmaxf(top, ws.ml[slots[j] * slot_rows + r0 + r].x);
        weight[j][r] = ws.unit[slots[j] * slot_rows + r0 + r];
      }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float less = top == -INFINITY ? 0.f : top;
    for (int j = l; j < parts; j += 16)
      if (slots[j] >= 0 && r < rows) {
        const float2 ml = ws.ml[slots[j] * slot_rows + r0 + r];
        const float f = ex2(ml.x - less);
        weight[j][r] *= f;
        sum = fmaf(ml.y, f, sum);
      }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum == 0.f ? 0.f : __fdividef(1.0f, sum);
    for (int j = l; j < parts; j += 16) weight[j][r] *= inv;  // (this thread's own)
    if (l == 0) row_ml[r] = make_float2(top, sum);
  }
  __syncthreads();
  // a thread's rows (r1 and on, kStep apart) go through the parts together, so that their loads are in flight together
  // (a prompt of 8192 tokens, 32 heads: 17 us, 20.5 one row after another)
  constexpr int kMost = kGroup * (kD / 4) / 256, kStep = 256 / (kD / 4);
  const int r1 = tid / (kD / 4), col = tid % (kD / 4);
  const float4* const part = reinterpret_cast<const float4*>(ws.o) + static_cast<size_t>(r0 + r1) * (kD / 4) + col;
  const auto add_up = [&](auto each) {
    constexpr int kEach = decltype(each)::value;
    if (r1 >= rows) return;
    float4 x[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = 0; j < parts; ++j) {
      if (slots[j] < 0) continue;
      const float4* const from = part + static_cast<size_t>(slots[j]) * slot_rows * (kD / 4);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        if (i > 0 && r1 + i * kStep >= rows) continue;
        const float4 y = from[i * kStep * (kD / 4)];
        const float f = weight[j][r1 + i * kStep];
        x[i].x = fmaf(y.x, f, x[i].x), x[i].y = fmaf(y.y, f, x[i].y);
        x[i].z = fmaf(y.z, f, x[i].z), x[i].w = fmaf(y.w, f, x[i].w);
      }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int r = r1 + i * kStep;
      if (r >= rows) continue;
      const float2 ml = row_ml[r];
      const AttnRow row = attn_row(p, s, cut.hk, cut.tile * kRows + r0 + r);
      if (!row_ok(p, row, kChkStore)) continue;
      *reinterpret_cast<uint2*>(p.o + row.at * kD + 4 * col) =
          make_uint2(pack_bf16x2(x[i].x, x[i].y), pack_bf16x2(x[i].z, x[i].w));
      if (col == 0 && p.lse != nullptr) p.lse[row.at] = attn_lse(ml.x, ml.y);
    }
  };
  if (rows > kStep)
    add_up(std::integral_constant<int, kMost>{});
  else
    add_up(std::integral_constant<int, 1>{});
}

}  // namespace coda
