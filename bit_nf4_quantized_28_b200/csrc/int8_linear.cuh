// int8_linear.cuh -- the linear in 8-bit integers that serves a merged weight:
//   y[t][n] = bf16( float(sum_k x[t][k] w[n][k]) * (xs[t] * ws[n]) ),
// x codes with one scale per token, w codes with one scale per output
// channel.  The sum is an exact int32 (|x|, |w| <= 128 and k < 2^17 keep it
// below 2^31), so neither a split along k nor its order changes the result;
// the scales are applied to it once, in fp32.
#pragma once

#include "common.cuh"

namespace qn {

constexpr int64_t kInt8MaxK = (int64_t{1} << 17) - 16;

struct Int8Params {
  const int8_t* x;       // [m, k]
  const float* xs;       // [m]
  const int8_t* w;       // [n, k]
  const float* ws;       // [n]
  __nv_bfloat16* y;      // [m, n]
  int64_t m, n, k;
};

// D[16 x 8] += A[16 x 32] B[32 x 8], signed 8-bit operands, 32-bit sums.
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kInt8VecThreads = 256;

// 16 output channels x 8 tokens per CTA; its 8 warps take the 64-wide steps
// of k in turn and add their sums in shared memory.  The weight rows are the
// A operand (two 16-byte loads per thread and step: 64 contiguous bytes of
// each of 16 rows), the tokens the B operand.  Within a step the order of k
// is permuted, alike for both operands, so that a thread's 16 bytes serve as
// its fragments as they are.
__global__ void __launch_bounds__(kInt8VecThreads) int8_vec_kernel(Int8Params p) {
  __shared__ int acc[8][16][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, t0 = static_cast<int64_t>(blockIdx.y) * 8;
  const int8_t* w0 = p.w + min(n0 + g, p.n - 1) * p.k;
  const int8_t* w1 = p.w + min(n0 + g + 8, p.n - 1) * p.k;
  const int8_t* xr = p.x + min(t0 + g, p.m - 1) * p.k;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int d[4] = {0, 0, 0, 0};
  for (int64_t k = warp * 64 + q * 16; k - q * 16 < p.k; k += 512) {
    const bool in = k < p.k;
    const uint4 a = in ? *reinterpret_cast<const uint4*>(w0 + k) : zero;
    const uint4 b = in ? *reinterpret_cast<const uint4*>(w1 + k) : zero;
    const uint4 x = in ? *reinterpret_cast<const uint4*>(xr + k) : zero;
    const uint32_t f0[4] = {a.x, b.x, a.y, b.y}, f1[4] = {a.z, b.z, a.w, b.w};
    mma_s8(d, f0, x.x, x.y);
    mma_s8(d, f1, x.z, x.w);
  }
  acc[warp][g][2 * q] = d[0];
  acc[warp][g][2 * q + 1] = d[1];
  acc[warp][g + 8][2 * q] = d[2];
  acc[warp][g + 8][2 * q + 1] = d[3];
  __syncthreads();
  if (threadIdx.x < 128) {
    const int r = threadIdx.x & 15, c = threadIdx.x >> 4;
    int s = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += acc[i][r][c];
    if (n0 + r < p.n && t0 + c < p.m)
      p.y[(t0 + c) * p.n + n0 + r] = __float2bfloat16_rn(__int2float_rn(s) * (p.xs[t0 + c] * p.ws[n0 + r]));
  }
}

}  // namespace qn
