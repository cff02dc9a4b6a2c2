// Matrix product in 8-bit integers for groups of few rows (decode): the
// product of mm_i8_tc.cu where it is a stream of weights with a few dot
// products per weight, and a 128-row tile would be mostly empty.
//
//   y[r, n] = s_r w_n sum_k q[r, k] W[g][n, k]      (then ReLU, or SwiGLU of two)
//
// A task is 16 weight rows (SwiGLU: 8 gate rows and the 8 up rows of the same
// features) times a pass of up to 8 NB rows of its group, as mma.sync m16n8k32
// in int32.  Each lane fetches with cp.async the 16-byte pieces of the weight
// rows that it will multiply itself, DEPTH units of 256 bytes ahead, into slots
// of its own: nothing is handed over, so the stream has no barriers.  A
// thread's 16 bytes of rows g and g + 8 and of token g's row are one A and one
// B operand for a permuted order of K.  Rows longer than 2048 bytes are split
// over the eight warps of a group, whose partial sums meet in shared memory;
// shorter ones go one task to a warp.  Sums are exact, so the split does not
// change the result.
//
// The tasks of a warp or group are a run of consecutive ones, so the rows of its
// tokens stay in L1.
//
// Bound by latency for one matrix (one launch, one round of tasks: 4096 x 4096
// takes 6.4 us against 2.6 us of reading), by HBM for long ones: 65536 x 2048
// and one row 24.6 us, 5.5 TB/s.
#include "mm_i8.cuh"

namespace moe {
namespace {

using namespace ptx;
using i8::silu_f;

constexpr int CW = 16, GW = 8;              // warps, and those that share a task of long rows
constexpr int CT = 32 * CW;
constexpr int UNIT = 256, SEG = 64, SEGS = UNIT / SEG;
constexpr int DEPTH = 3;
constexpr int UNIT_BYTES = 16 * UNIT;
constexpr int SOLO_BYTES = 2048;

struct FewMmParams {
  const int32_t *offsets;
  int G, rows_cap;
  int N, K, b_stride, mode;
  int nb;                                   // row blocks of a group's weights
  const int8_t *q;
  const float *xs;
  const int8_t *w0, *w1;
  const float *ws0, *ws1;
  void *out;
  int *status;
  int set_status;                           // write the status word (nothing else clears it)
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where a walk over the tasks first .. end - 1 stands: task = (group, pass, row block)
struct Walk {
  int task, end;
  int g, row0, rows, b;                     // the pass's rows
};

__device__ __forceinline__ void locate(Walk &w, const int32_t *off, const int32_t *start, int G, int nb, int pass_rows) {
  int lo = 0, hi = G;                       // largest g with start[g] <= task
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= w.task) lo = mid; else hi = mid;
  }
  const int local = w.task - start[lo], pass = local / nb;
  w.g = lo;
  w.b = local - pass * nb;
  w.row0 = off[lo] + pass * pass_rows;
  w.rows = min(pass_rows, off[lo + 1] - w.row0);
}

template <int NB>
struct __align__(16) Partial {
  int red[2][CW][NB][32][4];
};

template <int NB>
__global__ void __launch_bounds__(CT, 1) i8_few_gemm(const __grid_constant__ FewMmParams p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, c = lane & 3;
  uint8_t *ring_ptr = smem_raw + warp * DEPTH * UNIT_BYTES;
  Partial<NB> *part = reinterpret_cast<Partial<NB> *>(smem_raw + CW * DEPTH * UNIT_BYTES);
  int32_t *off = reinterpret_cast<int32_t *>(part + 1), *start = off + (kMaxExperts + 1);
  const int G = p.offsets ? p.G : 1, nb = p.nb;
  if (warp == 0) {
    const bool bad = warp_group_offsets(p.offsets, G, p.rows_cap, p.rows_cap, off, start,
                                        [nb](int cnt) { return (cnt + 8 * NB - 1) / (8 * NB) * nb; });
    if (blockIdx.x == 0 && lane == 0) {
      if (p.set_status) *p.status = bad ? kDevBadOffsets : 0;
      else if (bad) record_status(p.status, kDevBadOffsets);
    }
  }
  __syncthreads();
  const bool pairs = p.mode == I8_SWIGLU;
  const bool solo = p.K <= SOLO_BYTES;
  const int cols = pairs ? 8 : 16;
  // this warp's (group's) run of tasks
  const long long total = start[G];
  const int workers = solo ? gridDim.x * CW : gridDim.x * (CW / GW);
  const int me = solo ? blockIdx.x + gridDim.x * warp : blockIdx.x + gridDim.x * (warp / GW);
  const int first = (int)(total * me / workers), end = (int)(total * (me + 1) / workers);
  // and its segments of a row
  const int ns = (p.K + SEG - 1) / SEG;
  const int s0 = solo ? 0 : warp % GW * ns / GW, s1 = solo ? ns : (warp % GW + 1) * ns / GW;
  const int nseg = s1 - s0, nu = (nseg + SEGS - 1) / SEGS;
  const bool uneven = p.K % SEG != 0 && s1 == ns;
  const bool has_piece = p.K - (ns - 1) * SEG - c * 16 > 0;       // this lane's, of the row's last segment
  const int whole = (nseg - (uneven ? 1 : 0)) / SEGS;
  const uint32_t ring = smem_u32(ring_ptr) + lane * 16;

  // ---- the fetching end: DEPTH units ahead, one cp.async group per step
  Walk fw;
  fw.task = first;
  fw.end = end;
  int fu = 0;
  uint32_t issued = 0, used = 0;
  const int8_t *lo = nullptr, *hi = nullptr;
  bool has_lo = false, has_hi = false;
  auto aim = [&]() {                        // at task fw.task
    locate(fw, off, start, G, nb, 8 * NB);
    const size_t base = (size_t)fw.g * p.b_stride;
    const int r0 = fw.b * cols, n0 = min(8, p.N - r0), n1 = pairs ? n0 : min(8, p.N - r0 - 8);
    has_lo = lg < n0;
    has_hi = lg < n1;
    const size_t at = (size_t)s0 * SEG + c * 16;
    lo = p.w0 + (base + r0 + lg) * p.K + at;
    hi = (pairs ? p.w1 + (base + r0 + lg) * p.K : p.w0 + (base + r0 + 8 + lg) * p.K) + at;
  };
  if (first < end && nseg > 0) aim();
  auto step = [&]() {
    if (fw.task < fw.end && nseg > 0) {
      const uint32_t dst = ring + issued % DEPTH * UNIT_BYTES;
      const int n = min(SEGS, nseg - fu * SEGS) - (uneven && fu + 1 == nu && !has_piece ? 1 : 0);
#pragma unroll
      for (int s = 0; s < SEGS; ++s) {
        if (s < n && has_lo) cp_async16(dst + s * 1024, lo + s * SEG);
        if (s < n && has_hi) cp_async16(dst + s * 1024 + 512, hi + s * SEG);
      }
      lo += UNIT;
      hi += UNIT;
      ++issued;
      if (++fu == nu) {
        fu = 0;
        if (++fw.task < fw.end) aim();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < DEPTH; ++i) step();

  // ---- the products
  Walk w;
  w.end = end;
  uint32_t red_it = 0;
  for (w.task = first; w.task < end; ++w.task) {
    locate(w, off, start, G, nb, 8 * NB);
    const int8_t *bp[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
      bp[n] = p.q + (size_t)(w.row0 + min(lg + 8 * n, w.rows - 1)) * p.K + (size_t)s0 * SEG + c * 16;
    int acc[NB][2][4] = {};
    // scales of what this thread holds at the end (long rows: value number id
    // of the task, other warps from task to task)
    const int id = (threadIdx.x % (32 * GW) + 64 * red_it) % (32 * GW);
    const int col = w.b * cols + (solo ? lg : id & (cols - 1));
    float wsc[2] = {0.f, 0.f};
    const size_t sbase = (size_t)w.g * p.b_stride;
    if (col < p.N) {
      wsc[0] = __ldg(p.ws0 + sbase + col);
      if (pairs) wsc[1] = __ldg(p.ws1 + sbase + col);
    }
    if (solo && !pairs && col + 8 < p.N) wsc[1] = __ldg(p.ws0 + sbase + col + 8);
    for (int u = 0; u < nu; ++u) {
      const uint8_t *a = ring_ptr + used % DEPTH * UNIT_BYTES + lane * 16;
      auto product = [&](int s, const uint4(&b)[NB], bool cut) {
        uint4 l = *reinterpret_cast<const uint4 *>(a + s * 1024), h = *reinterpret_cast<const uint4 *>(a + s * 1024 + 512);
        if (cut) l = h = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma_s8(acc[n][0], l.x, h.x, l.y, h.y, b[n].x, b[n].y);
          mma_s8(acc[n][1], l.z, h.z, l.w, h.w, b[n].z, b[n].w);
        }
      };
      if (u < whole) {
        uint4 b[SEGS][NB];
#pragma unroll
        for (int s = 0; s < SEGS; ++s)
#pragma unroll
          for (int n = 0; n < NB; ++n) b[s][n] = __ldg(reinterpret_cast<const uint4 *>(bp[n] + s * SEG));
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll
        for (int s = 0; s < SEGS; ++s) product(s, b[s], false);
      } else {
        const int n_seg = min(SEGS, nseg - u * SEGS);
        const int left = p.K - (s0 + u * SEGS) * SEG - c * 16;       // bytes of the row from this lane's place on
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll 1
        for (int s = 0; s < n_seg; ++s) {
          const bool cut = left - s * SEG <= 0;
          uint4 b[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n)
            b[n] = cut ? make_uint4(0u, 0u, 0u, 0u) : __ldg(reinterpret_cast<const uint4 *>(bp[n] + s * SEG));
          product(s, b, cut);
        }
      }
#pragma unroll
      for (int n = 0; n < NB; ++n) bp[n] += UNIT;
      ++used;
      step();
    }
    auto store = [&](int tok, int cc, float v) {
      const size_t at = (size_t)(w.row0 + tok) * p.N + cc;
      if (p.mode == I8_F32) static_cast<float *>(p.out)[at] = v;
      else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
    };
    // value of output row f (pairs: with the up row f + 8) for token tok
    auto finish = [&](int tok, int cc, int v, int up, float ws, float wu) {
      if (tok >= w.rows || cc >= p.N) return;
      const float xs = __ldg(p.xs + w.row0 + tok);
      float y = (float)v * (xs * ws);
      if (pairs) y = silu_f(y) * ((float)up * (xs * wu));
      else if (p.mode == I8_RELU) y = y < 0.f ? 0.f : y;             // a NaN stays one
      store(tok, cc, y);
    };
    if (solo) {
      // accumulators 0, 1: row g, tokens 2c, 2c + 1; 2, 3: row g + 8
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int v = acc[n][0][i] + acc[n][1][i], v8 = acc[n][0][i + 2] + acc[n][1][i + 2];
          finish(8 * n + 2 * c + i, col, v, v8, wsc[0], wsc[1]);
          if (!pairs) finish(8 * n + 2 * c + i, col + 8, v8, 0, wsc[1], 0.f);
        }
    } else {
      int(*red)[NB][32][4] = &part->red[red_it & 1u][warp / GW * GW];
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *reinterpret_cast<int4 *>(red[warp % GW][n][lane]) =
            make_int4(acc[n][0][0] + acc[n][1][0], acc[n][0][1] + acc[n][1][1], acc[n][0][2] + acc[n][1][2],
                      acc[n][0][3] + acc[n][1][3]);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / GW), "n"(32 * GW) : "memory");
      ++red_it;
      auto sum = [&](int row, int tok) {
        const int ln = (row & 7) * 4 + ((tok & 7) >> 1), i = (tok & 1) + (row >> 3) * 2, n = tok >> 3;
        int v = 0;
#pragma unroll
        for (int q = 0; q < GW; ++q) v += red[q][n][ln][i];
        return v;
      };
      const int tok0 = id / cols, f = id & (cols - 1);
      // a thread's tokens: 32 (pairs) or 16 apart
      for (int tok = tok0; tok < w.rows; tok += 32 * GW / cols)
        finish(tok, col, sum(f, tok), pairs ? sum(f + 8, tok) : 0, wsc[0], wsc[1]);
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <int NB>
cudaError_t run(const FewMmParams &p, cudaStream_t s) {
  const size_t smem = (size_t)CW * DEPTH * UNIT_BYTES + sizeof(Partial<NB>) + sizeof(int32_t) * 2 * (kMaxExperts + 1);
  static_assert((size_t)CW * DEPTH * UNIT_BYTES + sizeof(Partial<NB>) + sizeof(int32_t) * 2 * (kMaxExperts + 1) <= 227 * 1024,
                "shared memory");
  cudaError_t err = cudaFuncSetAttribute(i8_few_gemm<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  launch_pdl(i8_few_gemm<NB>, sm_count(), CT, smem, s, p);
  return cudaGetLastError();
}

}  // namespace

// One to sixteen rows of one matrix, or up to 32 rows of several of which no
// more than eight meet in a group on average.  Against the 128-row tiles (us,
// weights from HBM): 1 row of 4096 x 4096 6.4 for 16.8, 16 rows 8.1 for 16.5,
// 64 rows 20.1 for 16.1; 1 row of 14336 x 4096 14.9 for 32.8, 32 rows 34.1 for
// 24.6; 8 groups of one row, 4096 x 2048, 15.5 for 24.8.  Many groups keep the
// tiles' copies in flight as well (128 groups of four rows, 768 x 2048: 41.7
// for 43.0), and without the bound on the rows a batch that falls into one
// group would read its weights once per eight rows.
bool mm_i8_is_few(const MmI8Args &a) {
  return a.rows_cap <= 16 || (a.offsets && a.rows_cap <= 32 && a.rows_cap <= 8LL * a.G);
}

cudaError_t launch_mm_i8_few(const MmI8Args &a, cudaStream_t s) {
  FewMmParams p;
  p.offsets = a.offsets;
  p.G = a.G;
  p.rows_cap = a.rows_cap;
  p.N = a.N;
  p.K = a.K;
  p.b_stride = a.b_stride;
  p.mode = a.mode;
  p.nb = a.mode == I8_SWIGLU ? (a.N + 7) / 8 : (a.N + 15) / 16;
  p.q = a.q;
  p.xs = a.xs;
  p.w0 = a.w0;
  p.w1 = a.w1;
  p.ws0 = a.ws0;
  p.ws1 = a.ws1;
  p.out = a.out;
  p.status = a.status;
  p.set_status = a.set_status;
  const int G = a.offsets ? a.G : 1;
  return a.rows_cap <= 8LL * G ? run<1>(p, s) : run<2>(p, s);
}

}  // namespace moe
