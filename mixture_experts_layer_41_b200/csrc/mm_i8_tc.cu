// Matrix product in 8-bit integers over ragged groups of rows, on the
// 5th-generation tensor cores (sm_100a).
//
//   acc[r, n] = sum_k q[r, k] W[g(r)][n, k]            int32, exact
//   y[r, n]   = acc * s_r * w_n                        one scale per row (token) and per output channel
//   MODE_RELU:   y = max(y, 0);   MODE_SWIGLU: y = silu(y_gate) * y_up
//
// Both operands are K-major int8.  The sums are exact (K < 131072), acc is
// rounded to fp32 once (2^-24), the scales are two fp32 products, and the
// result is rounded to bf16 once, or kept in fp32.
//
// Per CTA (one per SM, persistent over a static tile schedule of 128 x BN
// tiles, the row tiles of a group innermost so the CTAs in flight share
// weight tiles through L2):
//   warp 0      TMA producer: A 128 x 128 bytes and two B boxes of BN/2 rows
//               per stage, 128-byte swizzle (a stage is 128 K elements, four
//               K = 32 MMAs: twice the operations of a bf16 stage at the same
//               bytes);
//   warp 1      owns 2 BN columns of TMEM (two int32 accumulators) and issues
//               tcgen05.mma.kind::i8 (M = 128, N = BN, K = 32);
//   warps 2-5   epilogue: tcgen05.ld, scales, activation, store.  Each warp
//               keeps its own copy of the tile's channel scales in shared
//               memory, fetched while the accumulator is still being built.
// BN is 256 unless that leaves SMs without a tile (launch_mm_i8_tc).  K is not
// cut, so a few rows times a narrow matrix run on as many SMs as there are
// 128 x 64 tiles.
//
// A tile's rows past its group's end belong to the next group (or are
// zero-filled by TMA past the buffer); their results are never stored.
// Every mbarrier wait is bounded (moe_set_wait_timeout_ns); on expiry the
// thread records a status code, raises a CTA-wide abort flag, drains what it
// issued, and the CTA frees its TMEM and exits.
#include "mm_i8.cuh"

namespace moe {
namespace {

using namespace ptx;
using namespace i8;

constexpr int THREADS = 192;

template <int BN>
struct Shape {
  static constexpr int A_BYTES = BM * BK;
  static constexpr int BH_BYTES = BN / 2 * BK;
  static constexpr int STAGE_BYTES = A_BYTES + 2 * BH_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  // kind::i8: D s32, A s8, B s8, both K-major, N / 8 in bits 17-22, M / 16 in bits 24-28
  static constexpr uint32_t IDESC = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                                    ((uint32_t)(BM >> 4) << 24);
};

struct MmParams {
  uint64_t timeout_ns;
  const int32_t *offsets;   // [G+1] or nullptr (one group of `rows`)
  int G, rows, rows_cap;
  int N, b_stride, K;
  int mode;
  int n_tiles;
  const float *xs;          // [rows_cap]
  const float *ws0, *ws1;   // channel scales, group g's at g * b_stride
  void *out;                // [rows_cap, N] bf16, or fp32 with MODE_F32
  int *status;
};

template <int BN>
struct SharedState {
  uint64_t full[Shape<BN>::STAGES];
  uint64_t empty[Shape<BN>::STAGES];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int32_t off[kMaxExperts + 1];
  int32_t tile_start[kMaxExperts + 1];
  __align__(16) float scale[4][BN];   // per epilogue warp: the tile's channel scales, accumulator column order
};

template <int BN>
constexpr size_t smem_bytes() {
  return (size_t)Shape<BN>::STAGES * Shape<BN>::STAGE_BYTES + sizeof(SharedState<BN>) + 1024;
}

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum));
}

struct TileInfo {
  int g, row0, rows, n;
};

template <int BN>
__device__ __forceinline__ TileInfo decode_tile(const SharedState<BN> *st, int G, int tile) {
  int lo = 0, hi = G;   // largest g with tile_start[g] <= tile; tile_start[G] > tile
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (st->tile_start[mid] <= tile) lo = mid; else hi = mid;
  }
  TileInfo ti;
  ti.g = lo;
  const int local = tile - st->tile_start[lo];
  const int cnt = st->off[lo + 1] - st->off[lo];
  const int mt = (cnt + BM - 1) / BM;
  ti.n = local / mt;
  ti.row0 = st->off[lo] + (local % mt) * BM;
  ti.rows = min(BM, st->off[lo + 1] - ti.row0);
  return ti;
}

template <int BN>
__global__ void __launch_bounds__(THREADS, 1)
i8_grouped_gemm(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB0,
                const __grid_constant__ CUtensorMap mapB1, const MmParams p) {
  pdl_wait();
  using S = Shape<BN>;
  constexpr int STAGES = S::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t *tiles = smem_raw + pad;
  SharedState<BN> *st = reinterpret_cast<SharedState<BN> *>(tiles + (size_t)STAGES * S::STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.offsets ? p.G : 1;
  const bool swiglu = p.mode == I8_SWIGLU;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&st->full[s], 1);
      mbar_init(&st->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&st->acc_full[b], 1);
      mbar_init(&st->acc_empty[b], 4);
    }
    mbar_init(&st->drain, 1);
    st->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapA) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapB0) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapB1) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&st->tmem_base)),
                 "r"(S::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    const int n_tiles = p.n_tiles;
    const bool bad = warp_group_offsets(p.offsets, G, p.rows, p.rows_cap, st->off, st->tile_start,
                                        [n_tiles](int cnt) { return ((cnt + BM - 1) / BM) * n_tiles; });
    if (bad && lane == 0) record_status(p.status, kDevBadOffsets);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = st->tmem_base;
  const int total = st->tile_start[G];
  const int kb_n = (p.K + BK - 1) / BK;
  volatile int *abort_flag = &st->abort_flag;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const TileInfo ti = decode_tile(st, G, tile);
        const int b0 = ti.g * p.b_stride + ti.n * (swiglu ? BN / 2 : BN);
        const int b1 = swiglu ? b0 : b0 + BN / 2;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!wait_bounded(&st->empty[s], ph ^ 1u, abort_flag, p.status, kDevTimeoutProducer, p.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t *sa = tiles + (size_t)s * S::STAGE_BYTES;
          const uint32_t fb = smem_u32(&st->full[s]);
          mbar_expect_tx(&st->full[s], S::STAGE_BYTES);
          tma_load_2d(smem_u32(sa), &mapA, fb, kb * BK, ti.row0);
          tma_load_2d(smem_u32(sa + S::A_BYTES), &mapB0, fb, kb * BK, b0);
          tma_load_2d(smem_u32(sa + S::A_BYTES + S::BH_BYTES), &mapB1, fb, kb * BK, b1);
        }
      }
      // let the copies already issued land before the CTA goes away: all of them
      // have when the issuer used them, but it may have given up
      const uint32_t first = it > (uint32_t)STAGES ? it - STAGES : 0u;
      for (uint32_t i = first; i < it; ++i)
        if (!wait_drain(&st->full[i % STAGES], (i / STAGES) & 1u)) record_status(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const uint32_t buf = tcount & 1u, use = tcount >> 1;
        if (!wait_bounded(&st->acc_empty[buf], (use & 1u) ^ 1u, abort_flag, p.status, kDevTimeoutMma, p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dt = tmem_base + buf * BN;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!wait_bounded(&st->full[s], ph, abort_flag, p.status, kDevTimeoutMma, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(tiles + (size_t)s * S::STAGE_BYTES);
          const uint64_t da = sw128_desc(sa);
          const uint64_t db = sw128_desc(sa + S::A_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_i8(dt, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), S::IDESC, (kb | kk) != 0 ? 1u : 0u);
          tc_commit(&st->empty[s]);
        }
        if (!ok) break;
        tc_commit(&st->acc_full[buf]);
        ++tcount;
      }
      // every MMA this thread issued has completed once `drain` flips
      tc_commit(&st->drain);
      if (!wait_drain(&st->drain, 0u)) record_status(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                 // TMEM lane quarter of this warp
    const int rloc = q * 32 + lane;         // row of the tile this thread stores
    float *sc = st->scale[q];
    uint32_t tcount = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const TileInfo ti = decode_tile(st, G, tile);
      const uint32_t buf = tcount & 1u, use = tcount >> 1;
      const bool valid = rloc < ti.rows;
      const size_t row = (size_t)(ti.row0 + (valid ? rloc : 0));
      const int col0 = ti.n * (swiglu ? BN / 2 : BN);
      load_scales<BN>(sc, p.ws0, p.ws1, (size_t)ti.g * p.b_stride, p.mode, p.N, col0);
      const float xs = valid ? __ldg(p.xs + row) : 0.f;
      // the warp goes on together or not at all
      const bool ok = wait_bounded(&st->acc_full[buf], use & 1u, abort_flag, p.status, kDevTimeoutEpilogue, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      store_tile<BN>(tmem_base + buf * BN + ((uint32_t)(q * 32) << 16), sc, xs, p.mode, p.out, p.N, row, col0, valid);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st->acc_empty[buf]);
      ++tcount;
    }
  }

  tc_fence_before();
  __syncthreads();
  pdl_trigger();                         // tiles done: the next kernel may be scheduled
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::TMEM_COLS)
                 : "memory");
  }
}

template <int BN>
cudaError_t run(const MmI8Args &a, cudaStream_t s) {
  using S = Shape<BN>;
  CUtensorMap ma, mb0, mb1;
  const int G = a.offsets ? a.G : 1;
  const int b_rows = (G - 1) * a.b_stride + a.N;
  cudaError_t err = make_map_i8(&ma, a.q, (uint64_t)a.K, (uint64_t)a.rows_cap, BM);
  if (err == cudaSuccess) err = make_map_i8(&mb0, a.w0, (uint64_t)a.K, (uint64_t)b_rows, BN / 2);
  if (err == cudaSuccess) err = make_map_i8(&mb1, a.mode == I8_SWIGLU ? a.w1 : a.w0, (uint64_t)a.K, (uint64_t)b_rows,
                                            BN / 2);
  if (err != cudaSuccess) return err;
  MmParams p;
  p.timeout_ns = wait_timeout_ns();
  p.offsets = a.offsets;
  p.G = a.G;
  p.rows = a.rows_cap;
  p.rows_cap = a.rows_cap;
  p.N = a.N;
  p.b_stride = a.b_stride;
  p.K = a.K;
  p.mode = a.mode;
  p.n_tiles = a.mode == I8_SWIGLU ? (a.N + BN / 2 - 1) / (BN / 2) : (a.N + BN - 1) / BN;
  p.xs = a.xs;
  p.ws0 = a.ws0;
  p.ws1 = a.ws1;
  p.out = a.out;
  p.status = a.status;
  const long long upper = ((long long)(a.rows_cap + BM - 1) / BM + G) * p.n_tiles;
  const int sms = sm_count();
  const int grid = (int)(upper < sms ? upper : sms);
  err = cudaFuncSetAttribute(i8_grouped_gemm<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<BN>());
  if (err != cudaSuccess) return err;
  // (scheduled while the row quantisation ends, as the pairs' launch explains)
  launch_pdl(i8_grouped_gemm<BN>, grid, THREADS, smem_bytes<BN>(), s, ma, mb0, mb1, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mm_i8_tc(const MmI8Args &a, cudaStream_t s) {
  // the widest tile that gives every SM one, else the narrowest
  const int G = a.offsets ? a.G : 1;
  const long long m_tiles = (long long)(a.rows_cap + BM - 1) / BM + (G > 1 ? G / 2 : 0);
  auto tiles = [&](int bn) {
    const int w = a.mode == I8_SWIGLU ? bn / 2 : bn;
    return m_tiles * ((a.N + w - 1) / w);
  };
  const int sms = sm_count();
  if (tiles(256) >= sms) return run<256>(a, s);
  if (tiles(128) >= sms) return run<128>(a, s);
  return run<64>(a, s);
}

}  // namespace moe
