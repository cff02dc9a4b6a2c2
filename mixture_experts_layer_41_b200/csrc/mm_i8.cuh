// Pieces shared by the 8-bit products on the tensor cores: tile sizes, and the
// epilogue that turns 32-bit sums into scaled, activated rows.  Internal to
// the library.
#pragma once

#include "tc_ptx.cuh"

namespace moe {
namespace i8 {

constexpr int BM = 128;                       // accumulator rows of a CTA
constexpr int BK = 128;                       // 128 int8 = one swizzle row

// (moe_forward_few, which waits for its weights anyway, divides exactly: its h
// can differ by a bf16 step.)  The approximate quotient is within 2 ulp (0 past 2^126, where silu is below
// 2^-119); the IEEE one branches, and cost the product of 8192 x 28672 x 4096
// a sixth of its time in the epilogue
__device__ __forceinline__ float silu_f(float g) { return __fdividef(g, 1.f + __expf(-g)); }

// 32 consecutive outputs of a row from column col0 (columns >= N dropped);
// vectors where the row pitch keeps them aligned
__device__ __forceinline__ void store32(void *out, bool f32, size_t row, int N, int col0, const float (&y)[32]) {
  if (f32) {
    float *o = static_cast<float *>(out) + row * N + col0;
    if ((N & 3) == 0) {
#pragma unroll
      for (int v = 0; v < 8; ++v)
        if (col0 + 4 * v < N)
          *reinterpret_cast<float4 *>(o + 4 * v) = make_float4(y[4 * v], y[4 * v + 1], y[4 * v + 2], y[4 * v + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i < N) o[i] = y[i];
    }
  } else {
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out) + row * N + col0;
    if ((N & 7) == 0) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (col0 + 8 * v < N)
          *reinterpret_cast<uint4 *>(o + 8 * v) =
              make_uint4(pack_bf16x2(y[8 * v], y[8 * v + 1]), pack_bf16x2(y[8 * v + 2], y[8 * v + 3]),
                         pack_bf16x2(y[8 * v + 4], y[8 * v + 5]), pack_bf16x2(y[8 * v + 6], y[8 * v + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col0 + i < N) o[i] = __float2bfloat16_rn(y[i]);
    }
  }
}

// one warp: the channel scales of the tile's accumulator columns, from output
// column col0 of the group whose scales start at sbase (SwiGLU: gate columns,
// then the up columns of the same features)
template <int BN>
__device__ __forceinline__ void load_scales(float *sc, const float *ws0, const float *ws1, size_t sbase, int mode,
                                            int N, int col0) {
  __syncwarp();                             // the previous tile's scales have been read
#pragma unroll
  for (int i = 0; i < BN; i += 32) {
    const int j = i + (threadIdx.x & 31);   // accumulator column
    const bool up = mode == I8_SWIGLU && j >= BN / 2;
    const int col = col0 + (up ? j - BN / 2 : j);
    sc[j] = col < N ? __ldg((up ? ws1 : ws0) + sbase + col) : 0.f;
  }
  __syncwarp();
}

// one warp: its 32 accumulator rows at tb, scaled, activated and stored
template <int BN>
__device__ __forceinline__ void store_tile(uint32_t tb, const float *sc, float xs, int mode, void *out, int N,
                                           size_t row, int col0, bool valid) {
  using namespace ptx;
  if (mode == I8_SWIGLU) {
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += 32) {
      uint32_t g[32], u[32];
      tmem_ld32(tb + c, g);
      tmem_ld32(tb + BN / 2 + c, u);
      tmem_wait_ld();
      if (valid && col0 + c < N) {
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float gv = (float)(int)g[i] * (xs * sc[c + i]);
          const float uv = (float)(int)u[i] * (xs * sc[BN / 2 + c + i]);
          y[i] = silu_f(gv) * uv;
        }
        store32(out, false, row, N, col0 + c, y);
      }
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < BN; c += 32) {
      uint32_t a[32];
      tmem_ld32(tb + c, a);
      tmem_wait_ld();
      if (valid && col0 + c < N) {
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          y[i] = (float)(int)a[i] * (xs * sc[c + i]);
          if (mode == I8_RELU) y[i] = y[i] < 0.f ? 0.f : y[i];     // a NaN stays one
        }
        store32(out, mode == I8_F32, row, N, col0 + c, y);
      }
    }
  }
}

}  // namespace i8
}  // namespace moe
