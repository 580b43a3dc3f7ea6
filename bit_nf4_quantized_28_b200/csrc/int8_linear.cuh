// int8_linear.cuh -- the linear in 8-bit integers that serves a merged weight:
//   y[t][n] = bf16( float(sum_k x[t][k] w[n][k]) * (xs[t] * ws[n]) ),
// x codes with one scale per token, w codes with one scale per output
// channel.  The sum is an exact int32 (|x|, |w| <= 128 and k < 2^17 keep it
// below 2^31), so neither a split along k nor its order changes the result;
// the scales are applied to it once, in fp32.
#pragma once

#include "common.cuh"

namespace qn {

constexpr int64_t kInt8EndK = int64_t{1} << 17;      // k is below this

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

// Two products: a thread's 16 bytes of each of its two weight rows and of its token.
__device__ __forceinline__ void vec_step(int (&d)[4], const uint4& a, const uint4& b, const uint4& x) {
  const uint32_t f0[4] = {a.x, b.x, a.y, b.y}, f1[4] = {a.z, b.z, a.w, b.w};
  mma_s8(d, f0, x.x, x.y);
  mma_s8(d, f1, x.z, x.w);
}

constexpr int kInt8VecTokens = 8;
constexpr int kInt8VecUnroll = 4;

// A few generated tokens: the weight is read once and HBM bounds the product.
// 16 output channels x up to 8 tokens per CTA; its W warps take the 64-wide
// steps of k in turn and add their sums in shared memory.  The weight rows
// are the A operand (two 16-byte loads per thread and step: 64 contiguous
// bytes of each of 16 rows), the tokens the B operand.  Within a step the
// order of k is permuted, alike for both operands, so that a thread's 16
// bytes serve as its fragments as they are: the weight goes from memory to
// registers to the product, a group of four steps (128 bytes) in flight per
// thread, or two groups with W = 8.
//
// W = 8 (two CTAs per SM) while the CTAs fit two per SM, else W = 4 (five per
// SM), whose 740 slots take the 688 CTAs of 11008 channels at once.  Measured
// (one token): 11008 x 4096 9.5 us with W = 4, 10.8 with W = 8; 4096 x 11008
// 9.9 with W = 8, 10.8 with one group in flight, 13.7 with W = 4; one step in
// flight 17.6.  (A ring of asynchronous copies in shared memory, 4 to 12
// steps deep, over persistent CTAs measured 10.2 to 12.2 and 10.5 to 11.5.)
template <int W>
__global__ void __launch_bounds__(32 * W, W == 8 ? 2 : 5) int8_vec_kernel(Int8Params p) {
  constexpr int U = kInt8VecUnroll;
  __shared__ int acc[W][16][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int8_t* w0 = p.w + min(n0 + g, p.n - 1) * p.k;
  const int8_t* w1 = p.w + min(n0 + g + 8, p.n - 1) * p.k;
  const int8_t* xr = p.x + g * p.k;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int d[4] = {0, 0, 0, 0};
  const int kend = static_cast<int>(p.k);
  const bool tok = g < static_cast<int>(p.m);
  pdl_launch_dependents();
  pdl_wait_primary();
  struct Group {
    uint4 a[U], b[U], x[U];
  };
  auto fetch = [&](Group& f, int k) {
    if (k + 64 * W * (U - 1) + 64 <= kend) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int ku = k + 64 * W * u + q * 16;
        f.a[u] = *reinterpret_cast<const uint4*>(w0 + ku);
        f.b[u] = *reinterpret_cast<const uint4*>(w1 + ku);
        f.x[u] = tok ? *reinterpret_cast<const uint4*>(xr + ku) : zero;
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int ku = k + 64 * W * u + q * 16;
        const bool in = ku < kend;
        f.a[u] = in ? *reinterpret_cast<const uint4*>(w0 + ku) : zero;
        f.b[u] = in ? *reinterpret_cast<const uint4*>(w1 + ku) : zero;
        f.x[u] = in && tok ? *reinterpret_cast<const uint4*>(xr + ku) : zero;
      }
    }
  };
  auto use = [&](const Group& f) {
#pragma unroll
    for (int u = 0; u < U; ++u) vec_step(d, f.a[u], f.b[u], f.x[u]);
  };
  constexpr int kStep = 64 * W * U;
  if constexpr (W == 8) {                          // few CTAs: the next group is loaded before this one is used
    Group f0, f1;
    fetch(f0, warp * 64);
    for (int k = warp * 64; k < kend; k += 2 * kStep) {
      if (k + kStep < kend) fetch(f1, k + kStep);
      use(f0);
      if (k + kStep < kend) {
        if (k + 2 * kStep < kend) fetch(f0, k + 2 * kStep);
        use(f1);
      }
    }
  } else {
    for (int k = warp * 64; k < kend; k += kStep) {
      Group f;
      fetch(f, k);
      use(f);
    }
  }
  acc[warp][g][2 * q] = d[0];
  acc[warp][g][2 * q + 1] = d[1];
  acc[warp][g + 8][2 * q] = d[2];
  acc[warp][g + 8][2 * q + 1] = d[3];
  __syncthreads();
  const int r = threadIdx.x & 15, c = threadIdx.x >> 4;
  if (c < static_cast<int>(p.m) && n0 + r < p.n) {
    int s = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) s += acc[i][r][c];
    p.y[c * p.n + n0 + r] = __float2bfloat16_rn(__int2float_rn(s) * (p.xs[c] * p.ws[n0 + r]));
  }
}

}  // namespace qn
