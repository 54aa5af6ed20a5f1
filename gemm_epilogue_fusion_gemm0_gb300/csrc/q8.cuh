// q8.cuh -- the 8-bit operators' kernels: INT8 codes with scales.
//
// A value v is held as code * scale, code an integer in [-127, 127]:
//   scale = amax / 127,  code = rint(v * 127 / amax),  amax = max |v|
// over the values that share a scale: a row (a token), or 128 columns of a row
// (a checkpoint's block).  amax = 0 gives code 0 and scale 0; a row or block that
// holds an infinity or a NaN has the scale NaN, so that it stays visible in
// whatever the codes are used for.  The rounding to a code is off by at most
// amax / 254.
#pragma once

#include "epilogues.cuh"

namespace coda {

constexpr int kQ8Block = 128;  // columns per scale of a checkpoint

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(|a|, |b|, |c|), NaN if one of them is: one instruction
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}

__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16x2_2(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

// What a group of values with the given amax is multiplied by to give codes: 127 / amax to fp32's
// half ulp, from the approximate reciprocal and one correction by the exact remainder (an IEEE
// quotient costs a block of 128 values as much as the rest).
// Outside of 2^-100 .. 2^100 that quotient or its reciprocal leaves fp32's normal range, so the
// values are brought near one first (`pre`, a power of two: exact), which hardly any group needs.
struct Q8Factors {
  float pre, inv;
  __device__ __forceinline__ explicit Q8Factors(float amax) {
    pre = amax < 0x1p-100f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.0f;
    const float a = amax * pre;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    const float v = 127.0f * r;
    inv = amax > 0.f && amax <= 3.402823466e38f ? fmaf(fmaf(-v, a, 127.0f), r, v) : 0.f;
  }
  template <int kV>
  __device__ __forceinline__ void prepare(float (&u)[kV][8]) const {
    if (pre != 1.0f) {
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) u[v][e] *= pre;
    }
  }
};

// amax / 127: a product with the rounded 1 / 127, corrected once by its exact remainder
__device__ __forceinline__ float q8_scale(float amax) {
  const float s = amax * (1.0f / 127.0f);
  return amax <= 3.402823466e38f ? fmaf(fmaf(-127.0f, s, amax), 1.0f / 127.0f, s)
                                 : __int_as_float(0x7fffffff);
}

// Four codes of prepared values: v + 1.5 * 2^23 holds rint(v) (ties to even) in its low mantissa
// bits as a two's complement number for |v| < 2^22, so the code is the sum's low byte.
//
// kBf16: u and amax are bf16 numbers, whose codes are often half way between two integers (one in
// 400 of a bell-shaped tensor in blocks of 128).  The quotient's rounding would put such a code on
// either side, so the product is first rounded to multiples of 2^-15 (+ 1.5 * 2^8), which half
// way numbers are and which 127 * 2^-24, the quotient's error, does not leave.  All other
// codes >= 1/2 are further from half way than half of that step: with 8-bit mantissas a, b and
// v = a 2^-j, amax = b they are |254 a - (2 k + 1) 2^j b| / (2^(j+1) b) from it, j <= 8, the
// numerator even for j >= 1 and not 0: 2^-8 / 255 at least.  So a bf16 tensor's codes are the definition's.
// Other values (the norm's) go the shorter way, one rounding; theirs are off by 127 * 2^-24 and
// rarely half way.
template <bool kBf16>
__device__ __forceinline__ uint32_t q8_pack4(const float* u, const Q8Factors& f) {
  constexpr float kInt = 12582912.0f, kStep = 384.0f;  // 1.5 * 2^23, 1.5 * 2^8
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint64_t v = pack2(u[i], u[i + 1]), inv = pack2(f.inv, f.inv);
    float lo, hi;
    if constexpr (kBf16)
      unpack2(add2(fma2(v, inv, pack2(kStep, kStep)), pack2(kInt - kStep, kInt - kStep)), lo, hi);
    else
      unpack2(fma2(v, inv, pack2(kInt, kInt)), lo, hi);
    b[i] = __float_as_uint(lo);
    b[i + 1] = __float_as_uint(hi);
  }
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// the values of the four codes in a word, as fp32
__device__ __forceinline__ void q8_unpack4(uint32_t w, float (&v)[4]) {
  const int i = static_cast<int>(w);
  v[0] = static_cast<float>(i << 24 >> 24);
  v[1] = static_cast<float>(i << 16 >> 24);
  v[2] = static_cast<float>(i << 8 >> 24);
  v[3] = static_cast<float>(i >> 24);
}

// The same as two pairs: byte u = code + 128 under the exponent of 2^23 is 2^23 + u.  For epilogues,
// where the conversion instruction shares a slow unit with exponentials and reciprocals; the
// dequantiser, which has none, took 41 us this way instead of 33 (8192 x 8192).
__device__ __forceinline__ void q8_unpack4(uint32_t w, uint64_t (&v)[2]) {
  const uint32_t u = w ^ 0x80808080u;
  const auto at = [&](uint32_t sel) { return __uint_as_float(__byte_perm(u, 0x4b000000u, sel)); };
  const uint64_t less = pack2(-8388736.0f, -8388736.0f);  // 2^23 + 128
  v[0] = add2(pack2(at(0x7440), at(0x7441)), less);
  v[1] = add2(pack2(at(0x7442), at(0x7443)), less);
}

__device__ __forceinline__ void unpack8(const Chunk8& c, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf16lo(c.w[e]);
    v[2 * e + 1] = bf16hi(c.w[e]);
  }
}

// ---------------------------------------------------------------------------
// One scale per row: the plain quantiser (kNorm = false, u = x) and the RMS norm
// with the residual's addition (kNorm = true):
//   h = x + z,  r = 1 / sqrt(sum h^2 / d + eps),  norm = r h gamma = r u
// r is one positive number per row, so the codes rint(r u 127 / (r amax|u|)) do
// not need it: u's codes are the norm's, and the scale is r * amax|u| / 127.  One
// pass over the row therefore forms the sum of squares and the maximum together,
// the row waits in registers, and the codes follow.  h is used unrounded.
//
// Bound by HBM: 2 bytes in (4 with z), 1 out (3 with h) per value.  kVec vectors
// of 8 values per thread; a row belongs to a warp (kWarpRow, up to 1024 columns;
// 8 rows a block) or to a block of up to 1024 threads (up to 32768 columns).
// kVec = 0 is for longer rows: the second pass reads the row again.
// ---------------------------------------------------------------------------
struct RowQ8Params {
  const __nv_bfloat16* x;
  const __nv_bfloat16* z;      // may be null (kNorm)
  const __nv_bfloat16* gamma;  // kNorm
  __nv_bfloat16* h_out;        // may be null (kNorm)
  uint8_t* q_out;
  float* s_out;
  float eps;
  int M, d;
};

constexpr int kRowQ8Vec = 4;

// One vector of 8 values: h stored if wanted, u, and the row's sum of squares and maximum.
template <bool kNorm, bool kRes, bool kH, bool kPacked>
__device__ __forceinline__ void row_q8_values(const Chunk8& x, const Chunk8& z, const Chunk8& g,
                                              __nv_bfloat16* h_out, bool in, float (&u)[8],
                                              float& ss, float& amax) {
  unpack8(x, u);
  if constexpr (kNorm) {
    if constexpr (kRes) {
      float zv[8];
      unpack8(z, zv);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += zv[e];
    }
    if (kH && in) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(u[2 * e], u[2 * e + 1]);
      stg8(h_out, w);
    }
    float gv[8];
    unpack8(g, gv);
    if constexpr (kPacked) {
      uint64_t s2 = pack2(ss, 0.f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint64_t w = pack2(u[e], u[e + 1]);
        s2 = fma2(w, w, s2);
        unpack2(mul2(w, pack2(gv[e], gv[e + 1])), u[e], u[e + 1]);
      }
      float odd;
      unpack2(s2, ss, odd);
      ss += odd;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(u[e], u[e], ss);
        u[e] *= gv[e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; e += 2) amax = max3_abs_nan(amax, u[e], u[e + 1]);
}

template <bool kBf16>
__device__ __forceinline__ void q8_store8(uint8_t* q, const float (&u)[8], const Q8Factors& f) {
  *reinterpret_cast<uint2*>(q) = make_uint2(q8_pack4<kBf16>(u, f), q8_pack4<kBf16>(u + 4, f));
}

// kH: h is stored (h_out is not null)
template <bool kNorm, bool kRes, bool kH, int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) row_q8_kernel(const RowQ8Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = kWarpRow ? static_cast<int>(blockIdx.x) * 8 + warp : static_cast<int>(blockIdx.x);
  if (kWarpRow && row >= p.M) return;
  const int tid = kWarpRow ? lane : static_cast<int>(threadIdx.x);
  const int nthr = kWarpRow ? 32 : static_cast<int>(blockDim.x);
  // this thread's vectors of 8 values lie v * nthr past its first one, up to `last`
  const int last = p.d / 8 - 1 - tid;
  const size_t at = static_cast<size_t>(row) * p.d + 8 * tid;
  const __nv_bfloat16* const x = p.x + at;
  const __nv_bfloat16* const z = kRes ? p.z + at : nullptr;
  const __nv_bfloat16* const gm = kNorm ? p.gamma + 8 * tid : nullptr;
  __nv_bfloat16* const h = kH ? p.h_out + at : nullptr;
  uint8_t* const q = p.q_out + at;
  float ss = 0.f, amax = 0.f;
  float u[kVec > 0 ? kVec : 1][8];  // u, later prepared for its codes
  // Packed arithmetic where instructions are the bound (8192 x 264 with z 7.1 -> 6.1 us, 8192 x 5000
  // without 22.7 -> 22.1); not for a row of a block with z, which HBM bounds and whose loads it makes
  // the compiler spread out (8192 x 8192: 71 us, packed 76).
  constexpr bool kPacked = kWarpRow || !kRes;
  constexpr Chunk8 kZero = {{0u, 0u, 0u, 0u}};
  if constexpr (kVec > 0) {
    // All the loads first, without branches between them (a thread past the row's end reads
    // the row's last vector again, which its maximum does not mind and its sum leaves out): in
    // flight together.  With a branch around each vector the norm without a residual took
    // 55 us at 8192 x 8192.
    Chunk8 xr[kVec], zr[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int o = 8 * min(v * nthr, last);
      xr[v] = ldg8(x + o);
      zr[v] = kRes ? ldg8(z + o) : kZero;
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int o = 8 * min(v * nthr, last);
      const bool in = v * nthr <= last;
      float sv = 0.f;
      row_q8_values<kNorm, kRes, kH, kPacked>(xr[v], zr[v], kNorm ? ldg8(gm + o) : kZero, h + o, in, u[v], sv,
                                     amax);
      ss += in ? sv : 0.f;
    }
  } else {
    for (int i = 0; i <= last; i += nthr) {
      const size_t o = 8 * static_cast<size_t>(i);
      row_q8_values<kNorm, kRes, kH, kPacked>(ldg8(x + o), kRes ? ldg8(z + o) : kZero,
                                     kNorm ? ldg8(gm + o) : kZero, h + o, true, u[0], ss, amax);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (kNorm) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  if constexpr (!kWarpRow) {
    __shared__ float2 part[32];
    const int warps = nthr / 32;
    if (lane == 0) part[warp] = make_float2(ss, amax);
    __syncthreads();
    const float2 t = lane < warps ? part[lane] : make_float2(0.f, 0.f);
    ss = t.x;
    amax = t.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (kNorm) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
  }
  const Q8Factors f(amax);
  if (tid == 0) {
    const float s = q8_scale(amax);
    p.s_out[row] = kNorm ? s * rsqrtf(ss / static_cast<float>(p.d) + p.eps) : s;
  }
  if constexpr (kVec > 0) {
    f.prepare(u);
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (v * nthr <= last) q8_store8<!kNorm>(q + 8 * (v * nthr), u[v], f);
  } else {
    float s2 = 0.f, m2 = 0.f;
    for (int i = 0; i <= last; i += nthr) {
      const size_t o = 8 * static_cast<size_t>(i);
      row_q8_values<kNorm, kRes, false, kPacked>(ldg8(x + o), kRes ? ldg8(z + o) : kZero,
                                        kNorm ? ldg8(gm + o) : kZero, nullptr, true, u[0], s2, m2);
      f.prepare(u);
      q8_store8<!kNorm>(q + o, u[0], f);
    }
  }
}

// The same for many rows: blocks that stay and walk the rows, whose bytes arrive by bulk copies in a
// ring of `stages` rows in shared memory (gamma beside it), so that loads stay in flight while
// rows are reduced, quantised and stored and cost no registers.  A block per row, of which an SM holds
// one or two at these widths, keeps too few in flight: 8192 x 28672, norm without a residual 139 us
// and 108 here, the quantiser 133 and 120; 8192 x 20480, norm with one 171 and 142.
// Shared memory: [gamma | stages x (x row | z row) | barriers, abort flag].
constexpr int kRingMaxStages = 8;

__host__ __device__ __forceinline__ uint32_t row_ring_bytes(int d, bool norm, bool res, int stages) {
  return static_cast<uint32_t>((norm ? 1 : 0) + stages * (res ? 2 : 1)) * 2u *
             static_cast<uint32_t>(d) +
         8u * kRingMaxStages + 16u;
}

template <bool kNorm, bool kRes, bool kH>
__global__ void __launch_bounds__(1024) row_q8_ring_kernel(const RowQ8Params p, int stages,
                                                           uint64_t timeout_ns) {
  extern __shared__ __align__(128) uint8_t smem_ring[];
  __shared__ float2 part[2][32];
  constexpr int kVec = kRowQ8Vec;
  constexpr Chunk8 kZero = {{0u, 0u, 0u, 0u}};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tid = threadIdx.x, nthr = blockDim.x, warps = nthr / 32;
  const int nvec = p.d / 8;
  const uint32_t row_bytes = 2u * static_cast<uint32_t>(p.d);
  const uint32_t stage_bytes = (kRes ? 2u : 1u) * row_bytes;
  const uint32_t sG = smem_u32(smem_ring), ring = sG + (kNorm ? row_bytes : 0u);
  const uint32_t bar = ring + static_cast<uint32_t>(stages) * stage_bytes;
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(
      smem_ring + (bar - sG) + 8u * kRingMaxStages);
  const WaitCtl wc{timeout_ns, &g_coda_status, abort_flag};
  if (tid == 0) {
    *abort_flag = 0u;
    for (int s = 0; s < stages; ++s) mbar_init(bar + 8u * s, 1);
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();

  const int first = blockIdx.x, stride = gridDim.x;
  const int count = (p.M - 1 - first) / stride + 1;  // the grid has at most M blocks
  const auto issue = [&](int k) {                    // thread 0: this block's k-th row
    const uint32_t s = static_cast<uint32_t>(k % stages);
    const size_t at = static_cast<size_t>(first + static_cast<int64_t>(k) * stride) * p.d;
    mbar_arrive_expect_tx(bar + 8u * s, stage_bytes);
    bulk_load(ring + s * stage_bytes, p.x + at, row_bytes, bar + 8u * s);
    if (kRes) bulk_load(ring + s * stage_bytes + row_bytes, p.z + at, row_bytes, bar + 8u * s);
  };
  if (tid == 0)
    for (int k = 0; k < min(count, stages); ++k) issue(k);
  if constexpr (kNorm) {  // every thread reads back what it wrote itself
    for (int i = tid; i < nvec; i += nthr) {
      const Chunk8 g = ldg8(p.gamma + 8 * i);
      st_shared_v4(sG + 16u * i, g.w[0], g.w[1], g.w[2], g.w[3]);
    }
  }
  const auto lds8 = [](uint32_t addr) {
    const uint4 v = ld_shared_v4(addr);
    return Chunk8{{v.x, v.y, v.z, v.w}};
  };
  uint32_t s = 0, ph = 0;
  int k = 0;
  for (; k < count; ++k) {
    const int row = first + k * stride;
    const size_t base = static_cast<size_t>(row) * p.d;
    const bool ok = bounded_wait(bar + 8u * s, ph, wc, kSiteProducerEmpty);
    const uint32_t src = ring + s * stage_bytes;
    float u[kVec][8], ss = 0.f, amax = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = v * nthr + tid;
      if (i < nvec)
        row_q8_values<kNorm, kRes, kH, true>(lds8(src + 16u * i),
                                       kRes ? lds8(src + row_bytes + 16u * i) : kZero,
                                       kNorm ? lds8(sG + 16u * i) : kZero,
                                       kH ? p.h_out + base + 8 * static_cast<size_t>(i) : nullptr, true,
                                       u[v], ss, amax);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (kNorm) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (lane == 0) part[k & 1][warp] = make_float2(ss, amax);
    // also: every thread is done with the stage, and with the sums of the row before last
    if (!__syncthreads_and(ok)) break;
    if (tid == 0 && k + stages < count) issue(k + stages);
    const float2 t = lane < warps ? part[k & 1][lane] : make_float2(0.f, 0.f);
    ss = t.x;
    amax = t.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (kNorm) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    const Q8Factors f(amax);
    if (tid == 0) {
      const float sc = q8_scale(amax);
      p.s_out[row] = kNorm ? sc * rsqrtf(ss / static_cast<float>(p.d) + p.eps) : sc;
    }
    f.prepare(u);
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const int i = v * nthr + tid;
      if (i < nvec) q8_store8<!kNorm>(p.q_out + base + 8 * static_cast<size_t>(i), u[v], f);
    }
    if (++s == static_cast<uint32_t>(stages)) {
      s = 0;
      ph ^= 1u;
    }
  }
  if (k < count && tid == 0) land_copies(bar, min(count, k + stages), stages, timeout_ns);
}

// ---------------------------------------------------------------------------
// One scale per row and 128 columns.  A thread block's 256 threads cover up to 16
// neighbouring blocks of 128 columns of as many rows as that leaves (both powers of two:
// shifts, no division, which for so few values a thread would cost as much as the rest),
// several times, and all loads are issued before the first is used.
//
// Quantiser: a block belongs to 8 lanes of 16 values each, so its maximum is three
// shuffles away and nothing crosses a warp; the maximum is taken on packed bf16 pairs
// (exact: a maximum rounds nothing).  With 8 values a lane and IEEE quotients the
// work per block, not HBM, was the bound (8192 x 8192: 42 us, 72 %).
// Bound by HBM: 2 + 1 bytes per value and 4 per block.
// ---------------------------------------------------------------------------
constexpr int kQ8Passes = 4;

// log2 of the neighbouring blocks a thread block covers: nb rounded up to a power of two, 16 at most
__host__ __device__ __forceinline__ int q8_span_log2(int nb) {
  return nb > 8 ? 4 : nb > 4 ? 3 : nb > 2 ? 2 : nb > 1 ? 1 : 0;
}

// Where this thread's values of pass i are: row, block of the row, first column.  kLanes lanes
// share a block of 128 columns.
template <int kLanes>
struct Q8Place {
  static constexpr int kGroups = 256 / kLanes;  // blocks of 128 columns per pass
  int nb, blk, col, row0, rows_pass;
  bool in;  // the columns exist (the first 8 of them)
  __device__ __forceinline__ explicit Q8Place(int n) {
    nb = (n + kQ8Block - 1) / kQ8Block;
    const int lg = q8_span_log2(nb), gr = threadIdx.x / kLanes;
    rows_pass = kGroups >> lg;
    blk = (static_cast<int>(blockIdx.y) << lg) + (gr & ((1 << lg) - 1));
    col = blk * kQ8Block + kQ8Block / kLanes * static_cast<int>(threadIdx.x % kLanes);
    row0 = gr >> lg;
    in = blk < nb && col < n;
  }
  __device__ __forceinline__ int64_t row(int i) const {
    return (static_cast<int64_t>(blockIdx.x) * kQ8Passes + i) * rows_pass + row0;
  }
};

__device__ __forceinline__ uint32_t max2_nan_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

constexpr int kQ8QuantLanes = 8, kQ8DequantLanes = 16;

__global__ void __launch_bounds__(256) block_q8_kernel(const __nv_bfloat16* __restrict__ x,
                                                       uint8_t* __restrict__ q,
                                                       float* __restrict__ s, int M, int n) {
  griddep_launch_dependents();
  griddep_wait();
  const Q8Place<kQ8QuantLanes> pl(n);
  const bool in2 = pl.in && pl.col + 8 < n;  // n is a multiple of 8
  Chunk8 c[kQ8Passes][2];
#pragma unroll
  for (int i = 0; i < kQ8Passes; ++i) {
    const __nv_bfloat16* src = x + pl.row(i) * n + pl.col;
    const bool row_ok = pl.row(i) < M;
    c[i][0] = pl.in && row_ok ? ldg8(src) : Chunk8{{0u, 0u, 0u, 0u}};
    c[i][1] = in2 && row_ok ? ldg8(src + 8) : Chunk8{{0u, 0u, 0u, 0u}};
  }
#pragma unroll
  for (int i = 0; i < kQ8Passes; ++i) {
    uint32_t m2 = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m2 = max2_nan_bf16(m2, c[i][e / 4].w[e % 4] & 0x7fff7fffu);
    float amax = max_nan(bf16lo(m2), bf16hi(m2));
#pragma unroll
    for (int o = kQ8QuantLanes / 2; o > 0; o >>= 1)
      amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const Q8Factors f(amax);
    if (pl.row(i) < M) {
      uint8_t* dst = q + pl.row(i) * n + pl.col;
      float u[2][8];
      unpack8(c[i][0], u[0]);
      unpack8(c[i][1], u[1]);
      f.prepare(u);
      if (pl.in) q8_store8<true>(dst, u[0], f);
      if (in2) q8_store8<true>(dst + 8, u[1], f);
      if (threadIdx.x % kQ8QuantLanes == 0 && pl.in) s[pl.row(i) * pl.nb + pl.blk] = q8_scale(amax);
    }
  }
}

// Codes back to bf16: x = bf16(code * scale), the scale of the row (kRowScale) or of
// the row and 128 columns.  16 lanes of 8 values share a block; bound by HBM, 1 + 2 bytes.
template <bool kRowScale>
__global__ void __launch_bounds__(256) dequant_q8_kernel(const uint8_t* __restrict__ q,
                                                         const float* __restrict__ s,
                                                         __nv_bfloat16* __restrict__ x, int M,
                                                         int n) {
  griddep_launch_dependents();
  griddep_wait();
  const Q8Place<kQ8DequantLanes> pl(n);
  uint2 c[kQ8Passes];
  float sc[kQ8Passes];
#pragma unroll
  for (int i = 0; i < kQ8Passes; ++i) {
    const bool ok = pl.in && pl.row(i) < M;
    c[i] = ok ? __ldg(reinterpret_cast<const uint2*>(q + pl.row(i) * n + pl.col)) : make_uint2(0u, 0u);
    sc[i] = ok ? __ldg(s + (kRowScale ? pl.row(i) : pl.row(i) * pl.nb + pl.blk)) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kQ8Passes; ++i) {
    if (!pl.in || pl.row(i) >= M) continue;
    float lo[4], hi[4];
    q8_unpack4(c[i].x, lo);
    q8_unpack4(c[i].y, hi);
    const uint32_t o[4] = {pack_bf16x2(sc[i] * lo[0], sc[i] * lo[1]),
                           pack_bf16x2(sc[i] * lo[2], sc[i] * lo[3]),
                           pack_bf16x2(sc[i] * hi[0], sc[i] * hi[1]),
                           pack_bf16x2(sc[i] * hi[2], sc[i] * hi[3])};
    stg8(x + pl.row(i) * n + pl.col, o);
  }
}

// ---------------------------------------------------------------------------
// The INT8 product through the bf16 tensor cores.  sm_103a has no INT8 form of
// tcgen05.mma (ptxas refuses kind::i8 for it), and a code in [-128, 127] is
// exact in bf16 (8 significant bits), so the codes are multiplied as bf16
// integers with fp32 sums.  A product is at most 2^14, so sums are exact while
// they stay below 2^24 and are rounded as fp32 sums are above.
// ---------------------------------------------------------------------------
// Codes to bf16 integers, 16 per thread.
__global__ void __launch_bounds__(256) q8_to_bf16_kernel(const uint8_t* __restrict__ q,
                                                         __nv_bfloat16* __restrict__ x, size_t n16) {
  griddep_launch_dependents();
  griddep_wait();
  const size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n16) return;
  const uint4 c = __ldg(reinterpret_cast<const uint4*>(q) + i);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v[4];
    q8_unpack4(w[k], v);
    o[2 * k] = pack_bf16x2(v[0], v[1]);
    o[2 * k + 1] = pack_bf16x2(v[2], v[3]);
  }
  uint4* dst = reinterpret_cast<uint4*>(x) + 2 * i;
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// Epilogue: y = a_s[m] * w_s[n] * acc (+ z), one rounding to bf16.
struct EpiTokenChannelScale : EpiDefaultCols {
  static constexpr uint32_t kStageBytesPerWarp = Stage64::kBytes;  // z / y

  struct Params {
    const float* a_s;        // [M]
    const float* w_s;        // [N]
    const __nv_bfloat16* z;  // [M, N] or null
    __nv_bfloat16* y_out;    // [M, N]
  };

  static __device__ __forceinline__ void apply(const Params& p, const WaitCtl&, const TileCtx& c) {
    const int m = c.mb * kBM + c.row;
    const WarpRows wr(c);
    const size_t pitch = static_cast<size_t>(c.N) * 2;
    const float as = m < c.M ? __ldg(p.a_s + m) : 0.f;
#pragma unroll 1
    for (int ch = 0; ch < kHalfChunks; ++ch) {
      const int col = c.half * kHalfCols + ch * 32;
      const int n0 = c.n0 + col;
      const int valid = valid_bytes(n0, c.nend, 2);
      const size_t off = static_cast<size_t>(wr.row0) * c.N + n0;
      if (p.z != nullptr)
        Stage64::load(c.stage, p.z + off, pitch, wr.rows, valid, span(p.z, c.M, pitch));
      uint32_t v[32];
      tmem_ld32(c.taddr + col, v);
      tmem_ld_wait(v);
      uint32_t zr[16], yw[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) zr[i] = 0u;
      __syncwarp();
      if (p.z != nullptr) Stage64::get(c.stage, zr);
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float4 ws = n0 + 4 * g < c.nend && checked(n0 + 4 * g + 4 <= c.N, kChkLoad)
                              ? __ldg(reinterpret_cast<const float4*>(p.w_s + n0 + 4 * g))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        const float y0 = fmaf(as * __uint_as_float(v[4 * g]), ws.x, bf16lo(zr[2 * g]));
        const float y1 = fmaf(as * __uint_as_float(v[4 * g + 1]), ws.y, bf16hi(zr[2 * g]));
        const float y2 = fmaf(as * __uint_as_float(v[4 * g + 2]), ws.z, bf16lo(zr[2 * g + 1]));
        const float y3 = fmaf(as * __uint_as_float(v[4 * g + 3]), ws.w, bf16hi(zr[2 * g + 1]));
        yw[2 * g] = pack_bf16x2(y0, y1);
        yw[2 * g + 1] = pack_bf16x2(y2, y3);
      }
      Stage64::put(c.stage, yw);
      __syncwarp();
      Stage64::flush(c.stage, p.y_out + off, pitch, wr.rows, valid, span(p.y_out, c.M, pitch));
      __syncwarp();
    }
  }
};

// ---------------------------------------------------------------------------
// SwiGLU backward epilogue from an 8-bit checkpoint of the pre-activation: as
// EpiSwiGLUBackward (acc = da = dout @ W2^T), with y = [g | u] = code * scale, one
// scale per row and 128 columns of the whole row [g | u], and, optionally, the
// gated activation a = silu(g) u recomputed for the down projection's weight
// gradient, so that neither y nor a is kept between forward and backward.
// The codes cost 2 bytes per (g, u) pair where the saved bf16 pair costs 4.  Arithmetic on pairs of
// columns: 8192 x 14336 outputs, Dout = 4096 645 -> 628 us, 1024 336 -> 315 (bf16 form 625, 333).
// A thread's 128 columns lie in one block of the gate half and, since the up
// half starts at column `half` (a multiple of 16), in at most two blocks there.
// ---------------------------------------------------------------------------
struct EpiSwiGLUBackwardQ8 : EpiDefaultCols {
  static constexpr uint32_t kStageBytesPerWarp = 2 * Stage64::kBytes;  // g codes / dg; u codes / du

  struct Params {
    const uint8_t* y_q;     // [M, 2 * half] INT8 codes of the pre-activation [g | u]
    const float* y_s;       // [M, nb], nb = ceil(2 * half / 128)
    int nb;
    __nv_bfloat16* dy_out;  // [M, 2 * half]
    __nv_bfloat16* a_out;   // [M, half] or null
    float* spart;           // [2 * nt][M]
  };

  static __device__ __forceinline__ void apply(const Params& p, const WaitCtl&, const TileCtx& c) {
    const int m = c.mb * kBM + c.row;
    const WarpRows wr(c);
    const int half = c.N;  // the GEMM's output width is the gated width
    const size_t q_pitch = 2 * static_cast<size_t>(half), pitch = 2 * q_pitch;
    const size_t a_pitch = 2 * static_cast<size_t>(half);
    const uint32_t buf0 = c.stage, buf1 = c.stage + Stage64::kBytes;
    const int jh = c.n0 + c.half * kHalfCols;  // the thread's first column, a multiple of 128
    const int ub = (half + jh) / kQ8Block;     // block of the up half that column jh lies in
    const int u_next = (ub + 1) * kQ8Block - half;  // gated column at which the next block begins
    float sg = 0.f, su0 = 0.f, su1 = 0.f;
    if (m < c.M && jh < half) {
      const float* srow = p.y_s + static_cast<size_t>(m) * p.nb;
      if (checked(jh / kQ8Block < p.nb && ub < p.nb, kChkLoad)) {
        sg = __ldg(srow + jh / kQ8Block);
        su0 = __ldg(srow + ub);
        su1 = __ldg(srow + min(ub + 1, p.nb - 1));
      }
    }
    float ss = 0.f;
    const uint32_t lane = threadIdx.x & 31u;
    // The next chunk's codes are in flight while the current one is worked on (four 16-byte
    // registers; the bf16 form would need twice as many).
    const size_t rbase = static_cast<size_t>(wr.row0) * q_pitch;
    const Span q_span = span(p.y_q, c.M, q_pitch);
    uint4 gf[Stage32::kGroups], uf[Stage32::kGroups];
    const auto fetch = [&](int j0) {
      const int valid = valid_bytes(j0, c.nend, 1);
      Stage32::fetch(gf, p.y_q + rbase + j0, q_pitch, wr.rows, valid, q_span);
      Stage32::fetch(uf, p.y_q + rbase + half + j0, q_pitch, wr.rows, valid, q_span);
    };
    fetch(jh);
#pragma unroll 1
    for (int ch = 0; ch < kHalfChunks; ++ch) {
      const int col = c.half * kHalfCols + ch * 32;
      const int j0 = c.n0 + col;
      const int valid = valid_bytes(j0, c.nend, 2);
      const size_t row_off = rbase + j0;
      Stage32::deposit(buf0, gf);
      Stage32::deposit(buf1, uf);
      if (ch + 1 < kHalfChunks) fetch(j0 + 32);
      uint32_t v[32];
      tmem_ld32(c.taddr + col, v);
      tmem_ld_wait(v);
      mask_chunk(v, j0, c.nend);
      __syncwarp();
      uint32_t gq[8], uq[8], aw[16];
      Stage32::get(buf0, gq);
      Stage32::get(buf1, uq);
      __syncwarp();  // the stores below write where other lanes' codes were
#pragma unroll
      for (int g8 = 0; g8 < 4; ++g8) {  // 8 columns: one 16-byte group of a staged row
        const uint64_t one = pack2(1.f, 1.f);
        // u_next is a multiple of 16
        const float su = j0 + 8 * g8 < u_next ? su0 : su1;
        uint32_t dgw[4], duw[4];
#pragma unroll
        for (int w = 2 * g8; w < 2 * g8 + 2; ++w) {
          uint64_t gv[2], uv[2];
          q8_unpack4(gq[w], gv);
          q8_unpack4(uq[w], uv);
#pragma unroll
          for (int k = 0; k < 2; ++k) {  // two columns in packed arithmetic
            const uint64_t da = pack2(__uint_as_float(v[4 * w + 2 * k]),
                                      __uint_as_float(v[4 * w + 2 * k + 1]));
            const uint64_t g = mul2(pack2(sg, sg), gv[k]), u = mul2(pack2(su, su), uv[k]);
            float g0, g1, u0, u1, dg0, dg1, du0, du1;
            unpack2(g, g0, g1);
            unpack2(u, u0, u1);
            const uint64_t sig = pack2(__fdividef(1.0f, 1.0f + __expf(-g0)),
                                       __fdividef(1.0f, 1.0f + __expf(-g1)));
            // da u silu'(g), silu'(g) = sig (1 + g (1 - sig)), rounded as in the bf16 form
            const uint64_t dg = mul2(mul2(mul2(da, u), sig),
                                     fma2(g, fma2(sig, pack2(-1.f, -1.f), one), one));
            const uint64_t du = mul2(mul2(da, g), sig);
            unpack2(dg, dg0, dg1);
            unpack2(du, du0, du1);
            ss = fmaf(dg0, g0, ss);  // da is zero past the last row and column
            ss = fmaf(du0, u0, ss);
            ss = fmaf(dg1, g1, ss);
            ss = fmaf(du1, u1, ss);
            const int o = 2 * (w - 2 * g8) + k;
            dgw[o] = pack_bf16x2_2(dg);
            duw[o] = pack_bf16x2_2(du);
            aw[2 * w + k] = pack_bf16x2_2(mul2(mul2(g, sig), u));
          }
        }
        st_shared_v4(Stage64::at(buf0, lane, g8), dgw[0], dgw[1], dgw[2], dgw[3]);
        st_shared_v4(Stage64::at(buf1, lane, g8), duw[0], duw[1], duw[2], duw[3]);
      }
      __syncwarp();
      Stage64::flush(buf0, p.dy_out + row_off, pitch, wr.rows, valid, span(p.dy_out, c.M, pitch));
      Stage64::flush(buf1, p.dy_out + row_off + half, pitch, wr.rows, valid,
                     span(p.dy_out, c.M, pitch));
      __syncwarp();
      if (p.a_out != nullptr) {
        Stage64::put(buf0, aw);
        __syncwarp();
        Stage64::flush(buf0, p.a_out + static_cast<size_t>(wr.row0) * half + j0, a_pitch, wr.rows,
                       valid, span(p.a_out, c.M, a_pitch));
        __syncwarp();
      }
    }
    if (m < c.M && checked(partial_index(c, m) < static_cast<size_t>(2 * c.nt) * c.M, kChkPartial))
      p.spart[partial_index(c, m)] = ss;
  }
};

}  // namespace coda
