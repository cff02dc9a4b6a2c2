// Symmetric 8-bit row quantisation: one scale per row.
//
//   a = max_k |x_k|,  scale = a / 127,  code_k = rne(127 x_k / a)  in [-127, 127];
// a row of zeros has scale 0 and codes 0, a row that holds an infinity or a
// NaN has scale NaN and codes 0 (what is computed from it is then NaN, not a
// plausible number).
//
// The quotient is rounded as if it were exact, so the codes do not depend on
// how the division is done: a bf16 quotient is taken as p = t r (t = 127 x,
// exact; r = 1/a rounded), corrected once by its exact remainder t - p a.  The
// quotient can only equal n + 1/2 exactly, or miss it by more than 2^-17 of
// itself (both significands have 8 bits), and the corrected p is exact in the
// first case and within 2^-22 in the second; fp32 rows do the same in
// float64, where the smallest miss is 2^-32.  Rows whose largest element is
// very small or very large are scaled by a power of two first, so that
// neither r nor t leaves the normal range.
//
// Long rows are bound by HBM: each element is read once (a row stays in
// registers between the maximum and the codes) and each code written once.  A
// warp takes a row of up to 1024 elements, and of a matrix of many rows one of
// up to 4096 (fp32: 2048); a block of 256 threads one of up to 16384; longer rows are read a
// second time, from L2.  bf16, 8192 rows of 2048: 18.2 us (28.9 with a block to
// a row, whose two barriers every row waits for), 2.8 TB/s: bound by a warp's
// own chain of load, maximum, codes and store, with two blocks to an SM (119
// registers) beside it; 8192 of 14336: 68 us, 5.2 TB/s.
//
// The layer's use: rows of the expert-sorted matrix up to the device-side row
// count, or (scatter) token rows whose codes go straight to their slots' rows
// in expert order, which replaces the dispatch's copy at half its bytes.
#include "common.cuh"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int VECS = 8;       // 8-element vectors a thread keeps in registers
// rows from which a warp takes each.  us by blocks to by warps: bf16, 512 rows of
// 4096 3.8 to 5.9, 1024 6.4 to 6.6, 2048 10.9 to 9.3; fp32, 256 rows of 2048
// 2.8 (by blocks), 384 4.5 to 4.3, 777 6.8 to 4.8
constexpr int warp_rows_from(bool bf16) { return bf16 ? 1024 : 384; }

struct QuantParams {
  const void *x;
  long long rows;
  int K;                      // multiple of 16
  int8_t *q;
  float *scale;
  const int32_t *row_count;   // device: rows actually present (at most `rows`), or null
  const int32_t *slot_row;    // scatter: [rows, k] destination rows (-1: none), or null
  int k;
};

template <bool BF16>
struct Vec8 {
  uint32_t w[BF16 ? 4 : 8];
};

template <bool BF16>
__device__ __forceinline__ Vec8<BF16> load8(const void *x, size_t i) {
  Vec8<BF16> v;
  const uint4 a = __ldg(static_cast<const uint4 *>(x) + i * (BF16 ? 1 : 2));
  v.w[0] = a.x; v.w[1] = a.y; v.w[2] = a.z; v.w[3] = a.w;
  if constexpr (!BF16) {
    const uint4 b = __ldg(static_cast<const uint4 *>(x) + i * 2 + 1);
    v.w[4] = b.x; v.w[5] = b.y; v.w[6] = b.z; v.w[7] = b.w;
  }
  return v;
}

// largest |x| of the vector as fp32 bits (unsigned order: NaN above infinity)
template <bool BF16>
__device__ __forceinline__ uint32_t max8(const Vec8<BF16> &v, uint32_t m) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((v.w[i] << 16) & 0x7FFF0000u, v.w[i] & 0x7FFF0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7FFFFFFFu);
  }
  return m;
}

struct Row {
  float a, r;     // scaled maximum and its reciprocal
  double ad, rd;
  float pre;      // power of two the elements are scaled by
};

template <bool BF16>
__device__ __forceinline__ uint32_t code(float x, const Row &w) {
  if constexpr (BF16) {
    const float t = 127.f * (x * w.pre);
    const float p0 = t * w.r;
    const float p = __fmaf_rn(__fmaf_rn(-p0, w.a, t), w.r, p0);
    // adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and
    // leaves it in the low bits
    return __float_as_uint(p + 12582912.f);
  } else {
    const double t = 127.0 * (double)(x * w.pre);
    const double p0 = t * w.rd;
    const double p = __fma_rn(__fma_rn(-p0, w.ad, t), w.rd, p0);
    return (uint32_t)__double2loint(p + 6755399441055744.0);
  }
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

template <bool BF16>
__device__ __forceinline__ uint2 codes8(const Vec8<BF16> &v, const Row &w) {
  float f[8];
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v.w[i]);
  }
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code<BF16>(f[i], w);
  return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
}

// TPR threads per row (32 or THREADS), each with KEEP vectors in registers;
// MORE: rows longer than the registers hold
template <bool BF16, int TPR, int KEEP, bool MORE>
__global__ void __launch_bounds__(THREADS)
quantize_rows_kernel(const QuantParams p) {
  pdl_enter();
  __shared__ uint32_t red[THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i0 = TPR == 32 ? lane : threadIdx.x;
  const long long rows = p.row_count ? min((long long)max(*p.row_count, 0), p.rows) : p.rows;
  const int nv = p.K / 8;
  for (long long row = TPR == 32 ? (long long)blockIdx.x * (THREADS / 32) + warp : blockIdx.x; row < rows;
       row += TPR == 32 ? (long long)gridDim.x * (THREADS / 32) : gridDim.x) {
    const size_t base = (size_t)row * nv;
    Vec8<BF16> v[KEEP];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (i0 + j * TPR < nv) v[j] = load8<BF16>(p.x, base + i0 + j * TPR);
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (i0 + j * TPR < nv) m = max8<BF16>(v[j], m);
    if (MORE)
      for (int i = i0 + KEEP * TPR; i < nv; i += TPR) m = max8<BF16>(load8<BF16>(p.x, base + i), m);
    m = __reduce_max_sync(0xffffffffu, m);
    if (TPR != 32) {
      if (lane == 0) red[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) m = max(m, red[w]);
      __syncthreads();
    }
    const float a = __uint_as_float(m);
    Row w;
    w.pre = a < 0x1p-60f ? 0x1p64f : (a > 0x1p100f ? 0x1p-32f : 1.f);
    w.a = a * w.pre;
    if (m == 0u || m >= 0x7F800000u) {
      w.pre = 0.f;            // all codes 0 (0 * x is NaN for the bad rows: masked below)
      w.a = 1.f;
    }
    const bool bad = m >= 0x7F800000u;
    w.r = __frcp_rn(w.a);
    w.ad = BF16 ? 0.0 : (double)w.a;
    w.rd = BF16 ? 0.0 : 1.0 / w.ad;
    const float scale = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(a, 127.f);
    const int nd = p.slot_row ? p.k : 1;
    if (i0 == 0)
      for (int j = 0; j < nd; ++j) {
        const long long dst = p.slot_row ? p.slot_row[row * p.k + j] : row;
        if (dst >= 0) p.scale[dst] = scale;
      }
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int i = i0 + j * TPR;
      if (i < nv) {
        const uint2 c = bad ? make_uint2(0u, 0u) : codes8<BF16>(v[j], w);
        for (int s = 0; s < nd; ++s) {
          const long long dst = p.slot_row ? p.slot_row[row * p.k + s] : row;
          if (dst >= 0) reinterpret_cast<uint2 *>(p.q)[(size_t)dst * nv + i] = c;
        }
      }
    }
    if (MORE)
      for (int i = i0 + KEEP * TPR; i < nv; i += TPR) {
        const uint2 c = bad ? make_uint2(0u, 0u) : codes8<BF16>(load8<BF16>(p.x, base + i), w);
        for (int s = 0; s < nd; ++s) {
          const long long dst = p.slot_row ? p.slot_row[row * p.k + s] : row;
          if (dst >= 0) reinterpret_cast<uint2 *>(p.q)[(size_t)dst * nv + i] = c;
        }
      }
  }
}

template <bool BF16>
cudaError_t run(const QuantParams &p, cudaStream_t s) {
  constexpr int LONG = BF16 ? 16 : 8;       // vectors of a warp's lane in longer rows (64 registers)
  const bool warp_rows = p.K <= 4 * 32 * 8 || (p.K <= LONG * 32 * 8 && p.rows >= warp_rows_from(BF16));
  const long long blocks = warp_rows ? (p.rows + THREADS / 32 - 1) / (THREADS / 32) : p.rows;
  const int grid = (int)(blocks < 148 * 64 ? blocks : 148 * 64);
  if (p.K <= 4 * 32 * 8)
    launch_pdl(quantize_rows_kernel<BF16, 32, 4, false>, grid, THREADS, 0, s, p);
  else if (warp_rows)
    launch_pdl(quantize_rows_kernel<BF16, 32, LONG, false>, grid, THREADS, 0, s, p);
  else if (p.K <= VECS * THREADS * 8)
    launch_pdl(quantize_rows_kernel<BF16, THREADS, VECS, false>, grid, THREADS, 0, s, p);
  else
    launch_pdl(quantize_rows_kernel<BF16, THREADS, VECS, true>, grid, THREADS, 0, s, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_rows(const void *x, bool bf16, long long rows, int K, int8_t *q, float *scale,
                                 cudaStream_t s, const int32_t *row_count, const int32_t *slot_row, int k) {
  if (rows == 0) return cudaSuccess;
  const QuantParams p{x, rows, K, q, scale, row_count, slot_row, k};
  return bf16 ? run<true>(p, s) : run<false>(p, s);
}

}  // namespace moe
