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

// What a group of values with the given amax is multiplied by to give codes, as
// a product of two factors: 127 / amax overflows for amax below 127 / FLT_MAX, so
// such a group is brought up by `pre` = 2^100 first (exact: a power of two).
struct Q8Factors {
  float pre, inv;
  __device__ __forceinline__ explicit Q8Factors(float amax) {
    const bool tiny = amax < 0x1p-100f;
    pre = tiny ? 0x1p100f : 1.0f;
    inv = amax > 0.f ? 127.0f / (amax * pre) : 0.f;  // 0 for inf and NaN too
  }
};

__device__ __forceinline__ float q8_scale(float amax) {
  return amax <= 3.402823466e38f ? amax / 127.0f : __int_as_float(0x7fffffff);
}

// Four codes: v + 1.5 * 2^23 holds rint(v) (ties to even) in its low mantissa bits
// as a two's complement number for |v| < 2^22, so the code is the sum's low byte
// and one fused multiply-add rounds once.
__device__ __forceinline__ uint32_t q8_pack4(const float* u, const Q8Factors& f) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(fmaf(u[i] * f.pre, f.inv, 12582912.0f));
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

template <bool kNorm, bool kRes>
__device__ __forceinline__ void row_q8_load(const RowQ8Params& p, size_t base, int i, bool store_h,
                                            float (&u)[8], float& ss, float& amax) {
  unpack8(ldg8(p.x + base + 8 * static_cast<size_t>(i)), u);
  if constexpr (kNorm) {
    if constexpr (kRes) {
      float zv[8];
      unpack8(ldg8(p.z + base + 8 * static_cast<size_t>(i)), zv);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] += zv[e];
    }
    if (store_h) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(u[2 * e], u[2 * e + 1]);
      stg8(p.h_out + base + 8 * static_cast<size_t>(i), w);
    }
    float g[8];
    unpack8(ldg8(p.gamma + 8 * i), g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss = fmaf(u[e], u[e], ss);
      u[e] *= g[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(u[e]));
}

__device__ __forceinline__ void q8_store8(uint8_t* q, const float (&u)[8], const Q8Factors& f) {
  *reinterpret_cast<uint2*>(q) = make_uint2(q8_pack4(u, f), q8_pack4(u + 4, f));
}

template <bool kNorm, bool kRes, int kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) row_q8_kernel(const RowQ8Params p) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = kWarpRow ? static_cast<int>(blockIdx.x) * 8 + warp : static_cast<int>(blockIdx.x);
  if (kWarpRow && row >= p.M) return;
  const int tid = kWarpRow ? lane : static_cast<int>(threadIdx.x);
  const int nthr = kWarpRow ? 32 : static_cast<int>(blockDim.x);
  const int nvec = p.d / 8;
  const size_t base = static_cast<size_t>(row) * p.d;
  float ss = 0.f, amax = 0.f;
  float u[kVec > 0 ? kVec : 1][8];
  if constexpr (kVec > 0) {
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (v * nthr + tid < nvec)
        row_q8_load<kNorm, kRes>(p, base, v * nthr + tid, p.h_out != nullptr, u[v], ss, amax);
  } else {
    for (int i = tid; i < nvec; i += nthr)
      row_q8_load<kNorm, kRes>(p, base, i, p.h_out != nullptr, u[0], ss, amax);
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
  uint8_t* q = p.q_out + base;
  if constexpr (kVec > 0) {
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      if (v * nthr + tid < nvec) q8_store8(q + 8 * (v * nthr + tid), u[v], f);
  } else {
    float s2 = 0.f, m2 = 0.f;
    for (int i = tid; i < nvec; i += nthr) {
      row_q8_load<kNorm, kRes>(p, base, i, false, u[0], s2, m2);
      q8_store8(q + 8 * static_cast<size_t>(i), u[0], f);
    }
  }
}

// ---------------------------------------------------------------------------
// One scale per row and 128 columns.  A block of 128 columns belongs to 16 lanes
// of 8 values each, so its maximum is four shuffles away; nothing crosses a
// warp.  Blocks are numbered along the rows (the last one of a row may be
// ragged); a thread block takes 64 consecutive ones, four per half warp, whose
// loads are all issued before the first is used.  Bound by HBM: 2 + 1 bytes per
// value and 4 per block.
// ---------------------------------------------------------------------------
constexpr int kQ8Units = 4;                // blocks per half warp
constexpr int kQ8UnitsPerCta = 16 * kQ8Units;

// The half warp's units: unit `first + 16 i` as (row, block), i = 0, 1, ...
struct Q8Walk {
  size_t row;
  uint32_t blk;
  __device__ __forceinline__ Q8Walk(size_t unit, uint32_t nb) {
    row = unit / nb;
    blk = static_cast<uint32_t>(unit - row * nb);
  }
  __device__ __forceinline__ void next(uint32_t nb) {
    blk += 16;
    while (blk >= nb) {
      blk -= nb;
      ++row;
    }
  }
};

__global__ void __launch_bounds__(256) block_q8_kernel(const __nv_bfloat16* __restrict__ x,
                                                       uint8_t* __restrict__ q,
                                                       float* __restrict__ s, int M, int n) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t nb = static_cast<uint32_t>((n + kQ8Block - 1) / kQ8Block);
  const int sub = threadIdx.x & 15;
  const Q8Walk start(static_cast<size_t>(blockIdx.x) * kQ8UnitsPerCta + (threadIdx.x >> 4), nb);
  Chunk8 c[kQ8Units];
  Q8Walk w = start;
#pragma unroll
  for (int i = 0; i < kQ8Units; ++i, w.next(nb)) {
    const int col = static_cast<int>(w.blk) * kQ8Block + 8 * sub;
    c[i] = w.row < static_cast<size_t>(M) && col < n ? ldg8(x + w.row * n + col)
                                                     : Chunk8{{0u, 0u, 0u, 0u}};
  }
  w = start;
#pragma unroll
  for (int i = 0; i < kQ8Units; ++i, w.next(nb)) {
    float u[8], amax = 0.f;
    unpack8(c[i], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(u[e]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (w.row >= static_cast<size_t>(M)) continue;
    const Q8Factors f(amax);
    const int col = static_cast<int>(w.blk) * kQ8Block + 8 * sub;
    if (col < n) q8_store8(q + w.row * n + col, u, f);
    if (sub == 0) s[w.row * nb + w.blk] = q8_scale(amax);
  }
}

// Codes back to bf16: x = bf16(code * scale), the scale of the row (kRowScale) or of
// the row and 128 columns.  Work as in block_q8_kernel; bound by HBM, 1 + 2 bytes.
template <bool kRowScale>
__global__ void __launch_bounds__(256) dequant_q8_kernel(const uint8_t* __restrict__ q,
                                                         const float* __restrict__ s,
                                                         __nv_bfloat16* __restrict__ x, int M,
                                                         int n) {
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t nb = static_cast<uint32_t>((n + kQ8Block - 1) / kQ8Block);
  const int sub = threadIdx.x & 15;
  const Q8Walk start(static_cast<size_t>(blockIdx.x) * kQ8UnitsPerCta + (threadIdx.x >> 4), nb);
  uint2 c[kQ8Units];
  float sc[kQ8Units];
  Q8Walk w = start;
#pragma unroll
  for (int i = 0; i < kQ8Units; ++i, w.next(nb)) {
    const int col = static_cast<int>(w.blk) * kQ8Block + 8 * sub;
    const bool ok = w.row < static_cast<size_t>(M) && col < n;
    c[i] = ok ? __ldg(reinterpret_cast<const uint2*>(q + w.row * n + col)) : make_uint2(0u, 0u);
    sc[i] = ok ? __ldg(s + (kRowScale ? w.row : w.row * nb + w.blk)) : 0.f;
  }
  w = start;
#pragma unroll
  for (int i = 0; i < kQ8Units; ++i, w.next(nb)) {
    const int col = static_cast<int>(w.blk) * kQ8Block + 8 * sub;
    if (w.row >= static_cast<size_t>(M) || col >= n) continue;
    float lo[4], hi[4];
    q8_unpack4(c[i].x, lo);
    q8_unpack4(c[i].y, hi);
    const uint32_t o[4] = {pack_bf16x2(sc[i] * lo[0], sc[i] * lo[1]),
                           pack_bf16x2(sc[i] * lo[2], sc[i] * lo[3]),
                           pack_bf16x2(sc[i] * hi[0], sc[i] * hi[1]),
                           pack_bf16x2(sc[i] * hi[2], sc[i] * hi[3])};
    stg8(x + w.row * n + col, o);
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
// The codes cost 2 bytes per (g, u) pair where the saved bf16 pair costs 4.
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
        uint32_t dgw[4], duw[4];
#pragma unroll
        for (int w = 2 * g8; w < 2 * g8 + 2; ++w) {
          float gv[4], uv[4], dgv[4], duv[4], av[4];
          q8_unpack4(gq[w], gv);
          q8_unpack4(uq[w], uv);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float da = __uint_as_float(v[4 * w + k]);
            const float g = sg * gv[k];
            const float u = (j0 + 4 * w + k < u_next ? su0 : su1) * uv[k];
            const float sig = __fdividef(1.0f, 1.0f + __expf(-g));
            dgv[k] = da * u * sig * (1.0f + g * (1.0f - sig));
            duv[k] = da * g * sig;
            av[k] = g * sig * u;
            ss = fmaf(dgv[k], g, ss);  // da is zero past the last row and column
            ss = fmaf(duv[k], u, ss);
          }
          const int o = 2 * (w - 2 * g8);
          dgw[o] = pack_bf16x2(dgv[0], dgv[1]);
          dgw[o + 1] = pack_bf16x2(dgv[2], dgv[3]);
          duw[o] = pack_bf16x2(duv[0], duv[1]);
          duw[o + 1] = pack_bf16x2(duv[2], duv[3]);
          aw[2 * w] = pack_bf16x2(av[0], av[1]);
          aw[2 * w + 1] = pack_bf16x2(av[2], av[3]);
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
