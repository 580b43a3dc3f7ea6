// rmsnorm.cuh -- row-wise operators between the linears of a block: the RMS
// norm with the residual addition (bf16 out, its backward, or 8-bit out with
// one scale per row) and the quantization of rows to 8 bits.
//
// Forward:  h = bf16(x + res),  rstd = 1 / sqrt(mean(h^2) + eps),
//           y = bf16(h rstd w).
// 8 bits:   t = h w, amax = max |t| of the row, q = rint(127 t / amax),
//           scale = amax rstd / 127: q scale stands for h rstd w.  rstd is
//           positive and the same for the whole row, so it cancels in q: one
//           reduction over the row gives sum h^2 and amax together, where
//           quantizing y would need a second one behind the first.
//           t is exact in fp32 (two 8-bit significands) and so is 127 t, so
//           the codes do not depend on the order of any sum.
// Backward: g = dy w,  dx = dh + rstd (g - h rstd^2 mean(g h)),
//           dw = sum over rows of dy h rstd.
//
// HBM-bound: every element is read once and held in registers between the
// reduction and the output.  A CTA owns a row at a time; a thread holds NV
// vectors of 8 values (16-byte accesses), thread tid the vectors tid + i T.
#pragma once

#include "common.cuh"

namespace qn {

constexpr int kRowMaxNV = 8;
// most threads of a CTA: NV of 4 and 8 need more than the 64 registers that
// 1024 threads leave each
constexpr int row_max_threads(int nv) { return nv <= 2 ? 1024 : 512; }
constexpr int64_t kRowMaxCols = int64_t{8} * kRowMaxNV * row_max_threads(kRowMaxNV);

struct RowParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* res;   // kRes only
  const __nv_bfloat16* w;     // kNorm only
  __nv_bfloat16* h;           // kRes only
  __nv_bfloat16* y;           // bf16 output
  float* rstd;                // [m] or null (bf16 output)
  int8_t* q;                  // 8-bit output
  float* scale;               // [m]
  int64_t m;
  int d;
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sum and unsigned maximum over the CTA, to every thread, with one barrier.
// `buf` alternates between calls (two sets of 32 slots each), so that a warp
// may write the next row's values while another still reads this row's.
__device__ __forceinline__ void block_sum_max(float& s, uint32_t& a, float* fbuf, uint32_t* ubuf, int nw) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  a = __reduce_max_sync(0xFFFFFFFFu, a);
  if (lane == 0) {
    fbuf[warp] = s;
    ubuf[warp] = a;
  }
  __syncthreads();
  s = lane < nw ? fbuf[lane] : 0.f;
  a = lane < nw ? ubuf[lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  a = __reduce_max_sync(0xFFFFFFFFu, a);
}

// How a row with the given largest magnitude is brought to integers.  pre is
// a power of two that keeps 127 t and 127 / amax inside fp32's range; exact,
// so it changes no code.
struct RowScale {
  float pre;     // t is multiplied by this first
  float amax;    // pre * amax
  float inv;     // 127 / (pre * amax)
  bool fine;     // finite and not zero
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale s;
  const float a = __uint_as_float(amax_bits);
  s.fine = amax_bits != 0u && amax_bits < 0x7F800000u;
  s.pre = a > 0x1p100f ? 0x1p-32f : (a < 0x1p-60f ? 0x1p80f : 1.f);
  s.amax = s.fine ? a * s.pre : 1.f;
  s.inv = __fdiv_rn(127.f, s.amax);
  return s;
}

// rint(127 t / amax), the quotient rounded to fp32 first (ties to even).
// t * (127 / amax) is within 127 * 2^-23 < 2^-15 of it, so the division is
// needed only where that product lies within 2^-14 of a half-integer.
__device__ __forceinline__ int row_code(float t, const RowScale& s) {
  t *= s.pre;
  const float v = t * s.inv;
  float n = rintf(v);
  if (fabsf(fabsf(v - n) - 0.5f) < 0x1p-14f) n = rintf(__fdiv_rn(127.f * t, s.amax));
  return static_cast<int>(n);
}

template <int NV, bool kRes, bool kNorm, bool kInt8>
__global__ void __launch_bounds__(row_max_threads(NV)) row_kernel(RowParams p) {
  __shared__ float fbuf[2][32];
  __shared__ uint32_t ubuf[2][32];
  const int nvec = p.d >> 3;
  const int T = blockDim.x, nw = T >> 5;
  int par = 0;
  pdl_launch_dependents();
  pdl_wait_primary();
  for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x, par ^= 1) {
    const int64_t base = row * p.d;
    uint4 hv[NV];
    float ssq = 0.f;
    uint32_t amax = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      hv[i] = v < nvec ? *reinterpret_cast<const uint4*>(p.x + base + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (kRes) {
      uint4 rv[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * T;
        rv[i] = v < nvec ? *reinterpret_cast<const uint4*>(p.res + base + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * T;
        float a[8], b[8];
        unpack8(hv[i], a);
        unpack8(rv[i], b);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] += b[j];
        hv[i] = pack8(a);
        if (v < nvec) *reinterpret_cast<uint4*>(p.h + base + 8 * v) = hv[i];
      }
    }
    float t[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      unpack8(hv[i], t[i]);
      if constexpr (kNorm) {
        float wf[8];
        unpack8(v < nvec ? __ldg(reinterpret_cast<const uint4*>(p.w) + v) : make_uint4(0u, 0u, 0u, 0u), wf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ssq = fmaf(t[i][j], t[i][j], ssq);
          t[i][j] *= wf[j];
        }
      }
      if constexpr (kInt8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(t[i][j]) & 0x7FFFFFFFu);
      }
    }
    block_sum_max(ssq, amax, fbuf[par], ubuf[par], nw);
    const float rstd = kNorm ? __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ssq, static_cast<float>(p.d)) + p.eps)) : 1.f;
    if constexpr (kInt8) {
      const RowScale s = row_scale(amax);
      if (threadIdx.x == 0) {
        // a row with a non-finite value: its scale says so (NaN), its codes are 0
        const float a = __uint_as_float(amax);
        p.scale[row] = amax >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(kNorm ? a * rstd : a, 127.f);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * T;
        if (v >= nvec) continue;
        uint32_t o[2] = {0u, 0u};
        if (s.fine) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j >> 2] |= (static_cast<uint32_t>(row_code(t[i][j], s)) & 0xFFu) << (8 * (j & 3));
        }
        *reinterpret_cast<uint2*>(p.q + base + 8 * v) = make_uint2(o[0], o[1]);
      }
    } else {
      if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * T;
        if (v >= nvec) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) t[i][j] *= rstd;
        *reinterpret_cast<uint4*>(p.y + base + 8 * v) = pack8(t[i]);
      }
    }
  }
}

struct RowBwdParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* h;
  const __nv_bfloat16* w;
  const float* rstd;
  const __nv_bfloat16* dh;    // or null
  __nv_bfloat16* dx;
  float* part;                // kDw: [gridDim.x, d]
  int64_t m;
  int d;
};

template <int NV, bool kDw>
__global__ void __launch_bounds__(row_max_threads(NV)) row_bwd_kernel(RowBwdParams p) {
  __shared__ float fbuf[2][32];
  __shared__ uint32_t ubuf[2][32];
  const int nvec = p.d >> 3;
  const int T = blockDim.x, nw = T >> 5;
  const float inv_d = 1.f / static_cast<float>(p.d);
  float dw[kDw ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < (kDw ? NV : 1); ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  int par = 0;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  pdl_launch_dependents();
  pdl_wait_primary();
  for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x, par ^= 1) {
    const int64_t base = row * p.d;
    uint4 dyv[NV], hv[NV], av[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      dyv[i] = v < nvec ? *reinterpret_cast<const uint4*>(p.dy + base + 8 * v) : zero;
      hv[i] = v < nvec ? *reinterpret_cast<const uint4*>(p.h + base + 8 * v) : zero;
      av[i] = (p.dh && v < nvec) ? *reinterpret_cast<const uint4*>(p.dh + base + 8 * v) : zero;
    }
    const float rstd = p.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      float a[8], b[8], c[8];
      unpack8(dyv[i], a);
      unpack8(hv[i], b);
      unpack8(v < nvec ? __ldg(reinterpret_cast<const uint4*>(p.w) + v) : zero, c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kDw) dw[i][j] = fmaf(a[j], b[j] * rstd, dw[i][j]);
        dot = fmaf(a[j] * c[j], b[j], dot);
      }
    }
    uint32_t none = 0u;
    block_sum_max(dot, none, fbuf[par], ubuf[par], nw);
    const float c1 = dot * inv_d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      if (v >= nvec) continue;
      float a[8], b[8], c[8], e[8];
      unpack8(dyv[i], a);
      unpack8(hv[i], b);
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.w) + v), c);
      unpack8(av[i], e);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = fmaf(rstd, fmaf(-b[j], c1, a[j] * c[j]), e[j]);
      *reinterpret_cast<uint4*>(p.dx + base + 8 * v) = pack8(a);
    }
  }
  if constexpr (kDw) {
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * T;
      if (v >= nvec) continue;
      float4* o = reinterpret_cast<float4*>(out + 8 * v);
      o[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      o[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw = column sums of the CTAs' partial sums, in a fixed order.
__global__ void __launch_bounds__(256) row_dw_kernel(const float* part, float* dw, int rows, int d) {
  __shared__ float acc[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  pdl_launch_dependents();
  pdl_wait_primary();
  float s = 0.f;
  if (c < d)
    for (int r = warp; r < rows; r += 8) s += part[static_cast<int64_t>(r) * d + c];
  acc[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    for (int i = 1; i < 8; ++i) s += acc[i][lane];
    dw[c] = s;
  }
}

}  // namespace qn
