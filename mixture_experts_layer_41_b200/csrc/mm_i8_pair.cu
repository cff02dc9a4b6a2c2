// Matrix product in 8-bit integers over ragged groups of rows, on pairs of SMs
// (tcgen05 cta_group::2): the product of mm_i8_tc.cu for large groups, with
// the operands exchanged,
//
//   acc[n, r] = sum_k W[g][n, k] q[r, k].
//
// At twice the bf16 rate a 128 x 256 tile on one SM needs more of its shared
// memory than there is: each K = 32 step (128 clocks of tensor core) reads
// 12 KB of operands and receives 12 KB, at 128 bytes a clock.  A pair computes
// a 256 x 256 tile as one M = 256 MMA, each SM staging its own 128 weight rows
// and half of the token rows: 8 KB in and 8 KB out per step.  The weights are
// the M side because only N, the token side, can follow a group's size: its
// last tile has as many columns as it has rows, to a multiple of 64 (eight
// groups of about 1024 rows would pad 12 % with 256 of them as M).
//
// Per pair (persistent over a static tile schedule, the row tiles of a group
// innermost):
//   warp 0      TMA producer in both CTAs, 128-byte swizzle; the copies of
//               both complete on the even CTA's stage barrier, armed with the
//               bytes of both.  SwiGLU: 64 gate rows and the 64 up rows of the
//               same features to each CTA;
//   warp 1      both CTAs allocate 512 TMEM columns (two accumulators) as a
//               pair; the even CTA's lane 0 issues the MMAs and commits to
//               both CTAs' barriers at once;
//   warps 2-5   epilogue in both CTAs: a thread holds one output channel for
//               32 tokens at a time, and a warp stores 32 consecutive channels
//               of a token (64 bytes).  SwiGLU: the warps that hold a
//               feature's gate and up exchange half of their tokens in shared
//               memory.  The accumulator is released on the even CTA's barrier.
// No copy multicasts.
//
// Every mbarrier wait is bounded (moe_set_wait_timeout_ns); on expiry the
// thread records a status code, raises its CTA's abort flag and stops.  Either
// way the CTAs leave only when nothing comes to their shared memory any more
// (pair_leave), and free their TMEM.
#include "mm_i8.cuh"

namespace moe {
namespace {

using namespace ptx;
using namespace i8;

constexpr int BN = 256;                       // tokens of a full tile
constexpr int XBOX = 32;                      // rows of a copy in a group's last tile
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = BN / 2 * BK;          // this CTA's half of the token rows
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int THREADS = 192;
constexpr uint32_t TMEM_COLS = 512;
// kind::i8: D s32, A s8, B s8, both K-major, M / 16 in bits 24-28 (M = 256: the pair's rows); N / 8 goes to bits 17-22
constexpr uint32_t IDESC = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(2 * BM >> 4) << 24);

struct PairParams {
  uint64_t timeout_ns;
  const int32_t *offsets;   // [G+1] or nullptr (one group of rows_cap rows)
  int G, rows_cap;
  int N, b_stride, b_rows, K, n_tiles;
  const float *xs, *ws0, *ws1;
  void *out;
  int *status;
};

struct PairShared {
  uint64_t full[STAGES];     // even CTA: both CTAs' copies of a stage
  uint64_t empty[STAGES];    // every CTA: its stage is free again (pair commit)
  uint64_t acc_full[2];      // every CTA: an accumulator holds a finished tile
  uint64_t acc_empty[2];     // even CTA: both CTAs' epilogues have read it
  uint64_t drain;
  __align__(16) PairWork mine, theirs;
  uint32_t tmem_base;
  int abort_flag;
  int32_t off[kMaxExperts + 1];
  int32_t tile_start[kMaxExperts + 1];
  __align__(16) float xs[4][BN];        // per epilogue warp: the tile's token scales
  float swap[2][4][16][32];             // SwiGLU: the tokens a warp hands to its partner
  __align__(16) __nv_bfloat16 rows[4][32][32];   // per epilogue warp: 32 tokens' channels, on their way out
};

constexpr size_t SMEM_BYTES = (size_t)STAGES * STAGE_BYTES + sizeof(PairShared) + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accum) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accum));
}

struct PairTile {
  int g, row0, n;            // first token row, index of the weight rows
  int rows, cols;            // token rows, and accumulator columns (rows to a multiple of 64)
};

__device__ __forceinline__ PairTile decode_tile(const PairShared *st, int G, int tile) {
  int lo = 0, hi = G;        // largest g with tile_start[g] <= tile; tile_start[G] > tile
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (st->tile_start[mid] <= tile) lo = mid; else hi = mid;
  }
  PairTile t;
  t.g = lo;
  const int local = tile - st->tile_start[lo], cnt = st->off[lo + 1] - st->off[lo];
  const int row_tiles = (cnt + BN - 1) / BN, i = local % row_tiles;
  t.n = local / row_tiles;
  t.row0 = st->off[lo] + i * BN;
  t.rows = min(BN, cnt - i * BN);
  t.cols = (t.rows + 2 * XBOX - 1) / (2 * XBOX) * (2 * XBOX);
  return t;
}

// n tokens' 32 channels (this thread: f) from row `row` on, of which `left` are
// the tile's.  bf16 rows whose pitch keeps 16-byte vectors aligned go through
// the warp's part of shared memory, so that a store instruction writes eight
// rows' 64 bytes; others are stored element by element
template <int MODE, int n>
__device__ __forceinline__ void store_tokens(const PairParams &p, __nv_bfloat16 (*buf)[32], const float (&y)[n], int row,
                                             int left, int f) {
  const int lane = threadIdx.x & 31;
  if (MODE != I8_F32 && (p.N & 7) == 0) {
    __syncwarp();                           // the previous rows have been read
#pragma unroll
    for (int i = 0; i < n; ++i) buf[i][lane] = __float2bfloat16_rn(y[i]);
    __syncwarp();
    const int f8 = f - lane + lane % 4 * 8;
    if (f8 < p.N) {
      __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + (size_t)(row + lane / 4) * p.N + f8;
#pragma unroll
      for (int i = 0; i < n; i += 8, o += (size_t)8 * p.N)
        if (i + lane / 4 < left)
          *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(&buf[i + lane / 4][lane % 4 * 8]);
    }
  } else if (f < p.N) {
    const size_t at = (size_t)row * p.N + f;
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (i < left) {
        if (MODE == I8_F32) static_cast<float *>(p.out)[at + (size_t)i * p.N] = y[i];
        else static_cast<__nv_bfloat16 *>(p.out)[at + (size_t)i * p.N] = __float2bfloat16_rn(y[i]);
      }
  }
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
i8_pair_gemm(const __grid_constant__ CUtensorMap mapW0, const __grid_constant__ CUtensorMap mapW1,
             const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapXbox, const PairParams p) {
  pdl_wait();
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t *tiles = smem_raw + pad;
  PairShared *st = reinterpret_cast<PairShared *>(tiles + (size_t)STAGES * STAGE_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int G = p.offsets ? p.G : 1;
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  constexpr bool swiglu = MODE == I8_SWIGLU;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&st->full[s], 1);
      mbar_init(&st->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&st->acc_full[b], 1);
      mbar_init(&st->acc_empty[b], 8);          // 4 epilogue warps in each CTA
    }
    mbar_init(&st->drain, 1);
    st->abort_flag = 0;
    st->mine = {};
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapW0) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapW1) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)&mapX) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&st->tmem_base)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == 2) {
    const int n_tiles = p.n_tiles;
    const bool bad = warp_group_offsets(p.offsets, G, p.rows_cap, p.rows_cap, st->off, st->tile_start,
                                        [n_tiles](int cnt) { return (cnt + BN - 1) / BN * n_tiles; });
    if (bad && leader && lane == 0) record_status(p.status, kDevBadOffsets);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                        // both CTAs' barriers and TMEM exist before any use
  tc_fence_after();
  const uint32_t tmem_base = st->tmem_base;
  const int total = st->tile_start[G];
  const int kb_n = (p.K + BK - 1) / BK;
  volatile int *abort_flag = &st->abort_flag;
  const uint32_t full0 = map_to_rank(smem_u32(&st->full[0]), 0);        // the even CTA's barriers
  const uint32_t acc_empty0 = map_to_rank(smem_u32(&st->acc_empty[0]), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int tile = cluster; tile < total && ok; tile += n_clusters) {
        const PairTile ti = decode_tile(st, G, tile);
        // copies that would start past the last row are never used: they
        // fetch the first rows instead
        const int x0 = ti.row0 + (int)rank * (ti.cols / 2);
        int w0 = ti.g * p.b_stride + ti.n * (swiglu ? BM : 2 * BM) + (int)rank * (swiglu ? BM / 2 : BM);
        if (w0 >= p.b_rows) w0 = 0;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!wait_bounded<true>(&st->empty[s], ph ^ 1u, abort_flag, p.status, kDevTimeoutProducer, p.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t *sa = tiles + (size_t)s * STAGE_BYTES;
          const uint32_t fb = full0 + (uint32_t)(s * sizeof(uint64_t));
          if (leader) mbar_expect_tx(&st->full[s], 2 * (A_BYTES + ti.cols / 2 * BK));
          tma_load_2d_pair(smem_u32(sa), &mapW0, fb, kb * BK, w0);
          if (swiglu) tma_load_2d_pair(smem_u32(sa + A_BYTES / 2), &mapW1, fb, kb * BK, w0);
          if (ti.cols == BN) {
            tma_load_2d_pair(smem_u32(sa + A_BYTES), &mapX, fb, kb * BK, x0 < p.rows_cap ? x0 : 0);
          } else {
            for (int i = 0; i < ti.cols / 2; i += XBOX)
              tma_load_2d_pair(smem_u32(sa + A_BYTES + i * BK), &mapXbox, fb, kb * BK, x0 + i < p.rows_cap ? x0 + i : 0);
          }
        }
      }
      st->mine.issued = (int)it;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && leader) {
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = cluster; tile < total && ok; tile += n_clusters) {
        const uint32_t idesc = IDESC | ((uint32_t)(decode_tile(st, G, tile).cols >> 3) << 17);
        const uint32_t buf = tcount & 1u, use = tcount >> 1;
        if (!wait_bounded<true>(&st->acc_empty[buf], (use & 1u) ^ 1u, abort_flag, p.status, kDevTimeoutMma,
                                p.timeout_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t dt = tmem_base + buf * BN;
        for (int kb = 0; kb < kb_n; ++kb, ++it) {
          const int s = it % STAGES;
          const uint32_t ph = (it / STAGES) & 1u;
          if (!wait_bounded<true>(&st->full[s], ph, abort_flag, p.status, kDevTimeoutMma, p.timeout_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(tiles + (size_t)s * STAGE_BYTES);
          const uint64_t da = sw128_desc(sa);
          const uint64_t db = sw128_desc(sa + A_BYTES);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            tc_mma_pair(dt, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc, (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(&st->empty[s]);
        }
        if (!ok) break;
        tc_commit_pair(&st->acc_full[buf]);
        ++tcount;
      }
      // every MMA this thread issued has completed once `drain` flips
      tc_commit_pair(&st->drain);
      st->mine.committed = (int)it;
      st->mine.tiles = (int)tcount;
      if (!wait_drain<true>(&st->drain, 0u)) record_status(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;                 // TMEM lane quarter of this warp
    const int h = q >> 1;                   // SwiGLU: 0 holds gates, 1 the up values of warp q - 2's features
    const int bar = 1 + (q & 1);            // named barrier of the two
    float *xs = st->xs[q];
    uint32_t tcount = 0, swaps = 0;
    for (int tile = cluster; tile < total; tile += n_clusters) {
      const PairTile ti = decode_tile(st, G, tile);
      const uint32_t buf = tcount & 1u, use = tcount >> 1;
      // this thread's output channel and its scale
      const int f = swiglu ? ti.n * BM + (int)rank * (BM / 2) + (q & 1) * 32 + lane
                           : ti.n * 2 * BM + (int)rank * BM + q * 32 + lane;
      const float w = f < p.N ? __ldg((swiglu && h ? p.ws1 : p.ws0) + (size_t)ti.g * p.b_stride + f) : 0.f;
      __syncwarp();                         // the previous tile's scales have been read
      for (int j = lane; j < ti.rows; j += 32) xs[j] = __ldg(p.xs + ti.row0 + j);
      __syncwarp();
      bool ok = wait_bounded<true>(&st->acc_full[buf], use & 1u, abort_flag, p.status, kDevTimeoutEpilogue, p.timeout_ns);
      if (swiglu) {                         // the two warps go on together or not at all
        int both;
        asm volatile(
            "{\n\t.reg .pred p, r;\n\t"
            "setp.ne.s32 p, %1, 0;\n\t"
            "barrier.red.and.pred r, %2, 64, p;\n\t"
            "selp.s32 %0, 1, 0, r;\n\t}\n"
            : "=r"(both)
            : "r"((int)ok), "r"(bar)
            : "memory");
        ok = both != 0;
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + buf * BN + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < ti.rows; c += 32) {
        uint32_t a[32];
        tmem_ld32(tb + c, a);
        tmem_wait_ld();
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = (float)(int)a[i] * (xs[c + i] * w);
        if constexpr (!swiglu) {
          if (MODE == I8_RELU) {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = y[i] < 0.f ? 0.f : y[i];   // a NaN stays one
          }
          store_tokens<MODE, 32>(p, st->rows[q], y, ti.row0 + c, ti.rows - c, f);
        } else {
          float(*mine)[32] = st->swap[swaps & 1u][q], (*theirs)[32] = st->swap[swaps & 1u][q ^ 2];
          ++swaps;
#pragma unroll
          for (int j = 0; j < 16; ++j) mine[j][lane] = h ? y[j] : y[16 + j];
          asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
          float z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float o = theirs[j][lane];
            z[j] = silu_f(h ? o : y[j]) * (h ? y[16 + j] : o);
          }
          store_tokens<MODE, 16>(p, st->rows[q], z, ti.row0 + c + 16 * h, ti.rows - c - 16 * h, f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc_empty0 + buf * (uint32_t)sizeof(uint64_t));
      ++tcount;
    }
  }

  tc_fence_before();
  pair_leave<STAGES>(st->full, st->empty, st->acc_full, &st->drain, &st->mine, &st->theirs, abort_flag, p.status,
                     [&](int i) {
                       return (uint32_t)(A_BYTES + decode_tile(st, G, cluster + i / kb_n * n_clusters).cols / 2 * BK);
                     });
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                 : "memory");
  }
}

}  // namespace

// Groups of at least 192 rows, K of at least 1024, and more 128 x 64 tiles
// than SMs: what a pair saves in shared memory has to outweigh that there are
// fewer, larger tiles.  One SM to a pair, us: 4096 rows by 14336 x 4096 179.3
// to 163.4 (2.94 PFLOP/s), 1024 by 2048 x 4096 25.1 to 20.5, 8 groups of 1024
// by 4096 x 2048 65.7 to 59.6; on the other side 512 by 2048 x 4096 16.4 to
// 20.5, 1024 by 2048 x 512 9.5 to 12.3, 128 groups of four 152 to 157 in the
// layer that they are part of.
bool mm_i8_is_large(const MmI8Args &a) {
  const int G = a.offsets ? a.G : 1;
  const long long m_tiles = (long long)(a.rows_cap + BM - 1) / BM + G / 2;
  const int cols = a.mode == I8_SWIGLU ? 32 : 64;
  return a.K >= 1024 && a.rows_cap >= 192LL * G && m_tiles * ((a.N + cols - 1) / cols) > sm_count();
}

// Pairs resident at once (an SM left without a partner in its GPC takes no
// pair); 0 if that cannot be told
int mm_i8_pairs() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (sm_count() / 2), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  int n = 0;
  if (cudaFuncSetAttribute(i8_pair_gemm<I8_PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, i8_pair_gemm<I8_PLAIN>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_mm_i8_pair(const MmI8Args &a, int pairs, cudaStream_t s) {
  CUtensorMap mw0, mw1, mx, mxbox;
  const int G = a.offsets ? a.G : 1;
  const int b_rows = (G - 1) * a.b_stride + a.N;
  const bool swiglu = a.mode == I8_SWIGLU;
  const uint32_t w_box = swiglu ? BM / 2 : BM;
  cudaError_t err = make_map_i8(&mw0, a.w0, (uint64_t)a.K, (uint64_t)b_rows, w_box);
  if (err == cudaSuccess) err = make_map_i8(&mw1, swiglu ? a.w1 : a.w0, (uint64_t)a.K, (uint64_t)b_rows, w_box);
  if (err == cudaSuccess) err = make_map_i8(&mx, a.q, (uint64_t)a.K, (uint64_t)a.rows_cap, BN / 2);
  if (err == cudaSuccess) err = make_map_i8(&mxbox, a.q, (uint64_t)a.K, (uint64_t)a.rows_cap, XBOX);
  if (err != cudaSuccess) return err;
  PairParams p;
  p.timeout_ns = wait_timeout_ns();
  p.offsets = a.offsets;
  p.G = a.G;
  p.rows_cap = a.rows_cap;
  p.N = a.N;
  p.b_stride = a.b_stride;
  p.b_rows = b_rows;
  p.K = a.K;
  p.n_tiles = swiglu ? (a.N + BM - 1) / BM : (a.N + 2 * BM - 1) / (2 * BM);
  p.xs = a.xs;
  p.ws0 = a.ws0;
  p.ws1 = a.ws1;
  p.out = a.out;
  p.status = a.status;
  const long long upper = ((long long)(a.rows_cap + BN - 1) / BN + G) * p.n_tiles;
  auto kern = a.mode == I8_SWIGLU ? i8_pair_gemm<I8_SWIGLU>
              : a.mode == I8_RELU ? i8_pair_gemm<I8_RELU>
              : a.mode == I8_F32  ? i8_pair_gemm<I8_F32>
                                  : i8_pair_gemm<I8_PLAIN>;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (err != cudaSuccess) return err;
  const int clusters = (int)(upper < pairs ? upper : pairs);
  // (scheduled while the row quantisation ends: the 8-bit layer's step 1397 to
  // 1378 us at 4096 tokens, 547 to 539 at 8192 with one expert each, 34.3 to
  // 32.8 at 333)
  launch_pdl(kern, 2 * clusters, THREADS, SMEM_BYTES, s, mw0, mw1, mx, mxbox, p);
  return cudaGetLastError();
}

}  // namespace moe
