// attn_q8.cuh -- attention of new tokens over the 8-bit paged cache.
//
//   o[i] = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),  j <= lens - n + i
//   lse[i] = m_i + log sum_j p_ij
// i being one of a sequence's n new tokens, k_j and v_j the values of the cache's codes.  A row
// that sees no key is zero, its lse -inf.
#pragma once

#include "cache_q8.cuh"

namespace coda {

struct AttnQ8Params {
  const __nv_bfloat16* q;  // [rows, Hq, D]
  __nv_bfloat16* o;        // [rows, Hq, D]
  float* lse;              // [rows, Hq] or null
  CacheQ8 cache;
  BatchQ8 batch;
  int Hq, group;  // query heads; of them per key head
  float scale_log2;
};

// A warp per (row, query head): keys one after the other, the softmax's maximum and sum running.
template <int kD>
__global__ void __launch_bounds__(256) attn_q8_rows_kernel(const AttnQ8Params p) {
  constexpr int kE = kD / 32;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (u >= static_cast<int64_t>(p.batch.rows) * p.Hq) return;
  const int row = static_cast<int>(u / p.Hq), h = static_cast<int>(u % p.Hq), hk = h / p.group;
  const int b = sequence_of(p.batch, row, lane);
  if (b >= p.batch.B || row < __ldg(p.batch.cu)) return;
  // (the first token beyond the table's end makes the row NaN; none after it is walked)
  const int last = min(__ldg(p.batch.lens + b) - (__ldg(p.batch.cu + b + 1) - row),
                       p.batch.width << p.cache.page_log2);
  float q[kE], acc[kE] = {};
#pragma unroll
  for (int e = 0; e < kE; ++e) q[e] = __bfloat162float(p.q[u * kD + lane * kE + e]) * p.scale_log2;
  float m = -INFINITY, l = 0.f;
  int page = -1;
  for (int j = 0; j <= last; ++j) {
    const int slot = j & ((1 << p.cache.page_log2) - 1);
    if (slot == 0) page = page_of(p.batch, p.cache, b, j);
    float ks = __int_as_float(0x7fffffff), vs = ks;
    size_t e0 = 0;
    if (page >= 0) {
      e0 = cache_entry(p.cache, page, hk, slot);
      ks = p.cache.k_s[e0];
      vs = p.cache.v_s[e0];
    }
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      x += q[e] * static_cast<float>(static_cast<int8_t>(p.cache.k_q[e0 * kD + lane * kE + e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= ks;
    const float n = fmaxf(m, x), c = exp2f(m - n), w = exp2f(x - n);
    m = n;
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      acc[e] = acc[e] * c + w * vs * static_cast<float>(static_cast<int8_t>(p.cache.v_q[e0 * kD + lane * kE + e]));
  }
#pragma unroll
  for (int e = 0; e < kE; ++e)
    p.o[u * kD + lane * kE + e] = __float2bfloat16(last < 0 ? 0.f : acc[e] / l);
  if (p.lse != nullptr && lane == 0)
    p.lse[u] = last < 0 ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
}

}  // namespace coda
