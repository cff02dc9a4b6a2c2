// The whole layer for a few tokens (at most 16) in one cooperative kernel.
//
// Between two sampled tokens a server runs the layer on a handful of rows:
// nearly all of its time is reading the chosen experts' weights once.  The
// staged layer spends 9-10 launches on it and gives each weight tile a
// 128-row operand; here one persistent block per SM streams weight rows
// through shared memory without a pause, from the first product to the last.
//
//   router    each warp dots one expert's slice of the hidden dimension with
//             every token (fp32 products over runs of 8, float64 sums); the
//             shared expert's first product runs before anyone waits for it;
//   choice    after a grid barrier every block selects for all tokens from
//             the same partial sums (float64, ties to the lower expert) and
//             builds the same plan: per expert a 16-bit mask of its tokens in
//             token order, cut to the capacity;
//   phase 1   tasks of 16 weight rows: 8 gate rows and the 8 up rows of the
//             same features (ReLU: 16 rows), times the expert's tokens;
//   phase 2   tasks of 16 rows of the down projection, times h;
//   combine   after a last grid barrier: out = sum_j w_j y_j (+ shared).
//
// A block is one producer warp and eight consumer warps.  The producer copies
// rows, up to 2048 bytes of each of a task's 16 at a time, into a ring of stages
// (cp.async.bulk, one mbarrier per stage) and runs ahead of the consumers
// across tasks, phases and grid barriers: the ring is full of the next
// phase's weights when a barrier opens, and of the shared expert's while the
// router runs.  The row pitch in shared memory is 64 bytes more than a
// multiple of 128 (32 for 4-bit codes), so a warp reads its matrix fragments
// straight from the copied rows without bank conflicts.
// The consumers split a stage's K into 64-byte segments; per segment a thread
// takes 16 bytes of weight rows g and g + 8 and of token g's row, which is
// one A and one B operand of mma.sync m16n8 for a permuted order of K (a sum
// over K has no order).  mma.sync is the right unit here: 8 tokens are its N,
// and at a row of weights per 23 bytes a clock it is idle most of the time.
// The eight partial 16 x 8 results meet in shared memory.
//
// Precision: bf16 weights take h as the sum of two bf16 (16 bits); with 4-bit
// ones, whose products already keep the tensor pipe busy for most of the
// time a group of codes takes to arrive, h is one bf16, as in the staged
// layer.  4-bit codes are multiplied as exact small integers and scaled per
// group of 64 in fp32 (w = s q + b: s sum(q x) + b sum(x)).  Expert outputs
// stay fp32 until the combine.  8-bit weights follow
// the 8-bit layer's definition (rows of x and of the bf16 h quantised).
//
// Results do not depend on timing: every sum has a fixed order, and the row
// maxima behind the 8-bit codes of h are integer maxima.
// Bound by HBM.  All waits are bounded (moe_set_wait_timeout_ns): one that runs
// out records a status and turns every later wait of its block into a
// no-op, so the block runs through its (in-bounds) work, meets every barrier
// and ends.
#include "tc_ptx.cuh"

#include <math.h>

namespace moe {
namespace {

using namespace ptx;

constexpr int CW = 8;                       // consumer warps
constexpr int CT = 32 * CW;
constexpr int THREADS = CT + 32;
constexpr int MAX_CH = 2048;                // most bytes of a row per stage
constexpr int ROWS = 16;                    // weight rows per task
constexpr int MAX_STAGES = 24;
constexpr int MAX_SC = CW;                  // 4-bit: tasks whose scales and biases are held at once
constexpr int SC_BYTES = 64 * 1024;         // and the shared memory they may take (two tasks at least)
constexpr int MAX_T = kFewTokens;
constexpr int MAX_SLOTS = MAX_T * kMaxTopK;
constexpr int SMEM_LIMIT = 227 * 1024;

enum Fmt { BF16 = 0, I8 = 1, Q4 = 2 };

// row pitch in a stage beyond its ch bytes (a multiple of 128)
__host__ __device__ constexpr int pad_of(int fmt) { return fmt == Q4 ? 32 : 64; }

struct FewParams {
  uint64_t timeout_ns;
  int T, d, F, E, k, Fs;
  int router, norm;
  double scaling;
  int n_group, topk_group;
  int cap;                                  // slots an expert keeps, -1: all
  int swiglu;
  const uint16_t *x;
  const float *w_router, *bias;
  const void *w1, *w2, *w3;
  const void *s1, *s2, *s3, *b1, *b2, *b3;
  int w_stride;                             // w1 / w2 rows from one expert to the next
  const uint16_t *sw1, *sw2, *sw3;          // shared expert, bf16
  uint16_t *out;
  int32_t *ids;
  float *wts;
  int32_t *raw_counts, *kept_counts, *dropped;
  float *prob_sum;
  // workspace
  int *status;
  unsigned *bar;                            // grid barrier counters, zeroed before the launch
  double *logits;                           // [T][E]
  int8_t *xq;                               // 8-bit: [T][d] codes and scales of x
  float *xs;
  uint16_t *h;                              // [T*k][F], the low parts h_lo elements further
  size_t h_lo;
  uint16_t *hs;                             // [T][Fs] of the shared expert, likewise
  size_t hs_lo;
  unsigned *rowmax;                         // 8-bit: [T*k] largest |h| of a row, as fp32 bits
  int8_t *hq;                               // 8-bit: [T*k][F]
  float *y;                                 // [T*k + T][d] expert outputs, then the shared expert's
  int ch;                                   // bytes of a row per stage, a multiple of 128
  int stage_bytes, stages;
  int solo;                                 // warps that take tasks by themselves where rows are short
  int sc_slot, sc_slots;                    // 4-bit: bytes of one task's scales and biases, and how many are held
};

__host__ __device__ constexpr size_t scratch_bytes(int T, int E) { return ((size_t)T * E * 8 + 127) / 128 * 128; }

struct Shared {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t sc_full[MAX_SC], sc_empty[MAX_SC];
  uint64_t plan;
  int abort_flag;
  int nact;                                 // experts with rows
  uint32_t mask[kMaxExperts];               // tokens an expert keeps
  int16_t act[kMaxExperts];                 // the experts with rows
  int16_t row0[kMaxExperts + 1];            // first row of active expert i
  int sel_id[MAX_SLOTS];
  float sel_w[MAX_SLOTS];
  int16_t slot_row[MAX_SLOTS];
  int warp_n[CW], warp_rows[CW];            // per 32 experts: how many have rows, and the rows
  // partial results of the consumer warps, two tasks in turn
  __align__(16) uint32_t red[2][CW][2][32][4];
};

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(CT) : "memory"); }

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// ---------------------------------------------------------------- grid barrier
// Arrival and wait are apart, so work that does not depend on the other blocks
// can run between them.  Both are called by all consumer threads.
__device__ __forceinline__ void grid_arrive(unsigned *ctr) {
  consumer_sync();
  if (threadIdx.x == 0) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
  }
}
__device__ __forceinline__ void grid_wait(unsigned *ctr, volatile int *abort_flag, const FewParams &p) {
  if (threadIdx.x == 0) {
    const uint64_t t0 = global_ns();
    uint32_t spins = 0;
    for (;;) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      if (v >= gridDim.x || *abort_flag) break;
      if (((++spins & 31u) == 0 || p.timeout_ns < 1000u) && global_ns() - t0 > p.timeout_ns) {
        *abort_flag = 1;
        record_status(p.status, kDevTimeoutEpilogue);
        break;
      }
    }
    __threadfence();
  }
  consumer_sync();
}

// ---------------------------------------------------------------- tasks
// One task: 16 weight rows.  The order of a block's tasks is the same for the
// producer and the consumers: shared phase 1, shared phase 2, routed phase 1,
// routed phase 2.  Of each part a block takes a run of consecutive tasks, so
// most of them are one expert's and its tokens' rows stay in L1 (with tasks
// strided over the blocks every operand came from L2, and short rows waited for
// it); the blocks with one task more are others from part to part.  The shared expert needs no choice, so its weights
// stream while the router, the first barrier and the plan take their time.
enum Part { S1 = 0, S2 = 1, R1 = 2, R2 = 3 };

struct Dims {
  int nb;        // row blocks per expert
  int first, n;  // this block's tasks: first .. first + n - 1
};

__device__ __forceinline__ Dims part_dims(const FewParams &p, int part, int nact) {
  const int nbs1 = p.Fs / 8, nbs2 = p.Fs ? (p.d + ROWS - 1) / ROWS : 0;
  const int nb1 = p.swiglu ? p.F / 8 : (p.F + ROWS - 1) / ROWS, nb2 = (p.d + ROWS - 1) / ROWS;
  const int counts[4] = {nbs1, nbs2, nact * nb1, nact * nb2};
  const int nbs[4] = {nbs1, nbs2, nb1, nb2};
  const int G = (int)gridDim.x;
  int skip = 0;                              // blocks that already hold one task more
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < part) skip += counts[i] % G;
  const int b = ((int)blockIdx.x - skip % G + G) % G;
  const int q = counts[part] / G, rest = counts[part] % G;
  Dims r;
  r.nb = nbs[part];
  r.n = q + (b < rest ? 1 : 0);
  r.first = b * q + min(b, rest);
  return r;
}

template <int FMT>
__device__ __forceinline__ int row_bytes(int K) {
  return FMT == BF16 ? 2 * K : (FMT == I8 ? K : K / 2);
}

// Weight rows of a task: rows 0-7 from w0, 8-15 from w1, both `bytes` long
struct Src {
  const char *w0, *w1;
  int n0, n1;                               // valid rows of each half
  size_t r0, r1;                            // row index of each half's first (channel scales)
};

template <int FMT>
__device__ __forceinline__ Src task_src(const FewParams &p, int part, int e, int b) {
  Src s;
  if (part == S1 || part == R1) {
    const size_t base = part == S1 ? 0 : (size_t)e * p.w_stride;
    const size_t rb = row_bytes<FMT>(p.d);
    const char *g = static_cast<const char *>(part == S1 ? (const void *)p.sw1 : p.w1);
    const char *u = static_cast<const char *>(part == S1 ? (const void *)p.sw2 : p.w2);
    if (part == S1 || p.swiglu) {
      s.r0 = s.r1 = base + (size_t)b * 8;
      s.w0 = g + s.r0 * rb;
      s.w1 = u + s.r1 * rb;
      s.n0 = s.n1 = 8;
    } else {
      s.r0 = base + (size_t)b * ROWS;
      s.r1 = s.r0 + 8;
      s.w0 = g + s.r0 * rb;
      s.w1 = g + s.r1 * rb;
      s.n0 = min(8, p.F - b * ROWS);
      s.n1 = max(0, min(8, p.F - b * ROWS - 8));
    }
  } else {
    const size_t base = part == S2 ? 0 : (size_t)e * p.d;
    const size_t rb = row_bytes<FMT>(part == S2 ? p.Fs : p.F);
    const char *w = static_cast<const char *>(part == S2 ? (const void *)p.sw3 : p.w3);
    s.r0 = base + (size_t)b * ROWS;
    s.r1 = s.r0 + 8;
    s.w0 = w + s.r0 * rb;
    s.w1 = w + s.r1 * rb;
    s.n0 = min(8, p.d - b * ROWS);
    s.n1 = max(0, min(8, p.d - b * ROWS - 8));
  }
  return s;
}

// ---------------------------------------------------------------- producer
struct Ring {
  Shared *sh;
  uint8_t *tiles;
  uint8_t *sc;                              // 4-bit: the slots of scales and biases
  uint8_t *scratch;                         // [T][E] doubles: the tokens' probabilities
  uint32_t st, ph;                          // next stage and the parity of its use
  uint32_t sc_st, sc_ph;                    // likewise the next scale slot
  uint32_t issued, sc_issued;               // producer: copies' stages and slots so far
  bool ok;
};
__device__ __forceinline__ void advance(uint32_t &st, uint32_t &ph, uint32_t n) {
  if (++st == n) {
    st = 0;
    ph ^= 1u;
  }
}

// The slow half of a barrier wait, out of line
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *status, int code,
                                       uint64_t limit_ns) {
  return wait_bounded(bar, parity, abort_flag, status, code, limit_ns);
}
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, Shared *sh, const FewParams &p, int code) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, &sh->abort_flag, p.status, code, p.timeout_ns);
}

template <int FMT>
__device__ __forceinline__ void produce_part(const FewParams &p, Ring &r, int part, int nact) {
  const Dims dm = part_dims(p, part, nact);
  const int lane = threadIdx.x & 31;
  volatile int *abort_flag = &r.sh->abort_flag;
  const int K = part == S1 || part == R1 ? p.d : (part == S2 ? p.Fs : p.F);
  const int rb = row_bytes<FMT>(K);
  for (int task = dm.first; task < dm.first + dm.n && r.ok; ++task) {
    const int i = task / dm.nb, b = task - i * dm.nb;
    const Src s = task_src<FMT>(p, part, part == R1 || part == R2 ? r.sh->act[i] : 0, b);
    const bool mine = lane < 8 ? lane < s.n0 : (lane < ROWS && lane - 8 < s.n1);
    const char *row = lane < 8 ? s.w0 + (size_t)lane * rb : s.w1 + (size_t)(lane - 8) * rb;
    if (FMT == Q4) {
      // scales and biases of the task's two blocks of 8 rows, each contiguous
      int good = 1;
      if (lane == 0)
        good = wait_on(&r.sh->sc_empty[r.sc_st], r.sc_ph ^ 1u, r.sh, p, kDevTimeoutProducer) && !*abort_flag;
      if (!__shfl_sync(0xffffffffu, good, 0)) {
        r.ok = false;
        break;
      }
      const int blk = K / 64 * 2 * 8;       // bytes: a multiple of 16
      if (lane == 0) mbar_expect_tx(&r.sh->sc_full[r.sc_st], 4 * blk);
      __syncwarp();
      if (lane < 4) {
        const char *base = static_cast<const char *>(
            part == R2 ? (lane & 1 ? p.b3 : p.s3)
                       : (lane < 2 ? (lane & 1 ? p.b1 : p.s1) : (lane & 1 ? p.b2 : p.s2)));
        const size_t row_i = lane < 2 ? s.r0 : s.r1;
        bulk_load(smem_u32(r.sc + (size_t)r.sc_st * p.sc_slot + lane * blk), base + row_i * (size_t)(K / 64 * 2), blk,
                  smem_u32(&r.sh->sc_full[r.sc_st]));
      }
      ++r.sc_issued;
      advance(r.sc_st, r.sc_ph, p.sc_slots);
    }
    const uint32_t dst_row = smem_u32(r.tiles) + lane * (p.ch + pad_of(FMT));
    for (int off = 0; off < rb; off += p.ch) {
      int good = 1;
      if (lane == 0) {
        // a consumer that gave up releases stages it did not wait for, having
        // raised the flag first: nothing may be copied into them
        good = wait_on(&r.sh->empty[r.st], r.ph ^ 1u, r.sh, p, kDevTimeoutProducer) && !*abort_flag;
        if (good) mbar_expect_tx(&r.sh->full[r.st], min(p.ch, rb - off) * (s.n0 + s.n1));
      }
      if (!__shfl_sync(0xffffffffu, good, 0)) {
        r.ok = false;
        break;
      }
      if (mine)
        bulk_load(dst_row + r.st * p.stage_bytes, row + off, min(p.ch, rb - off), smem_u32(&r.sh->full[r.st]));
      ++r.issued;
      advance(r.st, r.ph, p.stages);
    }
  }
}

// ---------------------------------------------------------------- consumers
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// nibbles i and i + 4 of a code word as the exact bf16 pair (128 + q_i, 128 + q_{i+4})
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}
// 16 bytes of a token's row, kept in L1.  The rows that this kernel writes
// (codes of x, h) are read after a grid barrier, whose acquire keeps older
// copies out of L1.
__device__ __forceinline__ uint4 ld_l1(const char *p) {
  uint4 v;
  asm volatile("ld.global.ca.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// n arrivals at once
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
// the larger magnitude, NaN above all
__device__ __forceinline__ float abs_max(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
}
__device__ __forceinline__ uint4 lds128(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }

// B operand of one 64-byte segment of weight rows.  bf16 and 8-bit: 16 bytes
// of the token row (and of its low part).  4-bit: a segment is two groups of
// 64 codes; 16 elements of the token row per group.
template <int FMT, bool LO>
struct BSeg {
  uint4 v[FMT == Q4 ? 4 : 1][LO ? 2 : 1];
};

// segments whose operand a warp holds at once (4-bit: four times the registers each)
template <int FMT>
__host__ __device__ constexpr int segs_of() {
  return FMT == Q4 ? 2 : 4;
}

// bytes of the token row per byte of the weight row
template <int FMT>
__host__ __device__ constexpr int ratio_of() {
  return FMT == Q4 ? 4 : 1;
}

// row: this lane's place in the segment's stretch of the token row (its first
// byte plus lane_off); left: bytes of the weight row from the segment on.
// CHECK: the segment may reach past the row's end.
template <int FMT, bool LO, bool CHECK>
__device__ __forceinline__ void load_b(BSeg<FMT, LO> &bv, const char *row, size_t lo_bytes, int left, int c) {
#pragma unroll
  for (int q = 0; q < (FMT == Q4 ? 4 : 1); ++q) {
    // 4-bit: group q / 2 of the segment, elements 16 c + 8 (q % 2) ..
    constexpr int R = ratio_of<FMT>();
    const int at = FMT == Q4 ? (q >> 1) * 32 + (q & 1) * 4 : 0;
    const bool ok = !CHECK || at + c * (FMT == Q4 ? 8 : 16) < left;
#pragma unroll
    for (int l = 0; l < (LO ? 2 : 1); ++l)
      bv.v[q][l] = ok ? ld_l1(row + at * R + (l ? lo_bytes : 0)) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// Two accumulators per block of tokens, so that consecutive products do not
// wait for one another
template <int FMT, int NB>
struct Acc {
  float f[NB][2][4];
};
template <int NB>
struct Acc<I8, NB> {
  int f[NB][2][4];
};

// One 64-byte segment of the 16 rows times the tokens.  lo_row / hi_row: this
// lane's place in rows g and g + 8 (4-bit: without the lane's 8 c); left:
// bytes of the rows from the segment on.  sc: 4-bit, the group's scales of
// row g.  The first NBP blocks of eight tokens have their operand in
// registers; a further one (4-bit weights, whose operand is four times as
// long, and only for an expert that more than eight tokens chose) fetches it
// here from `far`.
template <int FMT, bool LO, int NB, int NBP, bool CHECK>
__device__ __forceinline__ void consume(Acc<FMT, NB> &acc, const BSeg<FMT, LO> (&bv)[NBP], const char *far, int left,
                                        const uint8_t *lo_row, const uint8_t *hi_row, bool second, int c,
                                        const uint16_t *sc, int groups) {
  if constexpr (FMT != Q4) {
    uint4 lo = lds128(lo_row), hi = lds128(hi_row);
    if (CHECK && c * 16 >= left) lo = hi = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (n > 0 && !second) break;
#pragma unroll
      for (int l = 0; l < (LO ? 2 : 1); ++l) {
        const uint4 b = bv[n].v[0][l];
        if constexpr (FMT == BF16) {
          mma_bf16(acc.f[n][0], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
          mma_bf16(acc.f[n][1], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
        } else {
          mma_s8(acc.f[n][0], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
          mma_s8(acc.f[n][1], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
        }
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (CHECK && q * 32 >= left) break;
      const uint2 lo = *reinterpret_cast<const uint2 *>(lo_row + q * 32);
      const uint2 hi = *reinterpret_cast<const uint2 *>(hi_row + q * 32);
      // scale and bias of rows g and g + 8 for this group.  The codes enter as
      // 128 + q (an exact bf16 by its bits), so the bias takes 128 s off again
      const float s_lo = bf16_to_f32(sc[q]), s_hi = bf16_to_f32(sc[16 * groups + q]);
      const float b_lo = fmaf(-128.f, s_lo, bf16_to_f32(sc[8 * groups + q]));
      const float b_hi = fmaf(-128.f, s_hi, bf16_to_f32(sc[24 * groups + q]));
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (n > 0 && !second) break;
        BSeg<FMT, LO> own;
        if (n >= NBP) load_b<FMT, LO, CHECK>(own, far, 0, left, c);
        float dq[4] = {0.f, 0.f, 0.f, 0.f}, dx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t wl = u ? lo.y : lo.x, wh = u ? hi.y : hi.x;
          constexpr uint32_t one = 0x3F803F80u;
          // elements (i, i + 4) of the token's 8, in the order of the nibble pairs
          const uint4 b = n < NBP ? bv[n < NBP ? n : 0].v[2 * q + u][0] : own.v[2 * q + u][0];
          const uint32_t p0 = __byte_perm(b.x, b.z, 0x5410), p1 = __byte_perm(b.x, b.z, 0x7632);
          const uint32_t p2 = __byte_perm(b.y, b.w, 0x5410), p3 = __byte_perm(b.y, b.w, 0x7632);
          mma_bf16(dq, code_pair(wl, 0), code_pair(wh, 0), code_pair(wl, 1), code_pair(wh, 1), p0, p1);
          mma_bf16(dx, one, one, one, one, p0, p1);
          mma_bf16(dq, code_pair(wl, 2), code_pair(wh, 2), code_pair(wl, 3), code_pair(wh, 3), p2, p3);
          mma_bf16(dx, one, one, one, one, p2, p3);
        }
        float(&a)[4] = acc.f[n][q];
        a[0] = fmaf(s_lo, dq[0], fmaf(b_lo, dx[0], a[0]));
        a[1] = fmaf(s_lo, dq[1], fmaf(b_lo, dx[1], a[1]));
        a[2] = fmaf(s_hi, dq[2], fmaf(b_hi, dx[2], a[2]));
        a[3] = fmaf(s_hi, dq[3], fmaf(b_hi, dx[3], a[3]));
      }
    }
  }
}

__device__ __forceinline__ float silu_f(float g) { return g / (1.f + expf(-g)); }

// n-th set bit of a mask (the mask has more than n)
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (int i = 0; i < n; ++i) m &= m - 1;
  return __ffs(m) - 1;
}

struct Cursor {
  int task, e, rows, row0, b;               // row0: first row of h / y
  uint32_t mask;
};

template <int PART>
__device__ __forceinline__ void place(const FewParams &p, const Shared *sh, const Dims &dm, Cursor &cu) {
  const int i = cu.task / dm.nb;
  cu.b = cu.task - i * dm.nb;
  if (PART == S1 || PART == S2) {
    cu.e = 0;
    cu.mask = (1u << p.T) - 1u;
    cu.row0 = 0;
    cu.rows = p.T;
  } else {
    cu.e = sh->act[i];
    cu.mask = sh->mask[cu.e];
    cu.row0 = sh->row0[i];
    cu.rows = sh->row0[i + 1] - cu.row0;
  }
}

// Row r of a task's token operand.  A row past the task's last repeats the
// last: each token is a column of its own, and those columns are not stored.
template <int FMT, int PART>
__device__ __forceinline__ const char *b_row(const FewParams &p, const Cursor &cu, int r) {
  r = min(r, cu.rows - 1);
  if (PART == S1 || PART == R1) {
    const int t = PART == S1 ? r : nth_bit(cu.mask, r);
    return FMT == I8 ? reinterpret_cast<const char *>(p.xq + (size_t)t * p.d)
                     : reinterpret_cast<const char *>(p.x + (size_t)t * p.d);
  }
  if (PART == S2) return reinterpret_cast<const char *>(p.hs + (size_t)r * p.Fs);
  return FMT == I8 ? reinterpret_cast<const char *>(p.hq + (size_t)(cu.row0 + r) * p.F)
                   : reinterpret_cast<const char *>(p.h + (size_t)(cu.row0 + r) * p.F);
}

// What becomes of one finished value: row f of the task's `cols` (with its up
// projection u where the task holds pairs), token tok.  Returns the magnitude
// of the stored bf16 h (8-bit weights: the row maxima are taken from it).
template <int FMT, int PART>
__device__ __forceinline__ float emit(const FewParams &p, const Cursor &cu, int f, int tok, float v, float u) {
  constexpr bool PHASE2 = PART == S2 || PART == R2;
  const bool pairs = PART == S1 || (PART == R1 && p.swiglu);
  const int col = cu.b * (pairs ? 8 : ROWS) + f;
  const int N = PART == S1 ? p.Fs : (PART == R1 ? p.F : p.d);
  if (tok >= cu.rows || col >= N) return 0.f;
  const size_t row = (size_t)cu.row0 + tok;
  if (FMT == I8) {
    // row scale: of the token (phase 1), of the row of h (phase 2)
    float xs;
    if (PHASE2) {
      const uint32_t top = __ldcg(p.rowmax + row);
      xs = top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(top), 127.f);
    } else {
      xs = __ldcg(p.xs + nth_bit(cu.mask, tok));
    }
    const size_t r0 = (size_t)cu.e * (PHASE2 ? p.d : p.w_stride) + col;
    v *= xs * __ldg(static_cast<const float *>(PHASE2 ? p.s3 : p.s1) + r0);
    if (pairs) u *= xs * __ldg(static_cast<const float *>(p.s2) + r0);
  }
  if (PHASE2) {
    p.y[(PART == S2 ? (size_t)p.T * p.k + tok : row) * p.d + col] = v;
    return 0.f;
  }
  if (pairs) v = silu_f(v) * u;
  else v = v < 0.f ? 0.f : v;               // a NaN stays one
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  uint16_t *h = PART == S1 ? p.hs + (size_t)tok * p.Fs + col : p.h + row * p.F + col;
  *h = *reinterpret_cast<const uint16_t *>(&hi);
  if (FMT == BF16) {
    const float rest = v - __bfloat162float(hi);
    const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
    h[PART == S1 ? p.hs_lo : p.h_lo] = *reinterpret_cast<const uint16_t *>(&lo);
  }
  return __bfloat162float(hi);
}

// The block's tasks of one part.  Long rows: the eight warps split each
// stage's K, and their partial results meet in shared memory.  SOLO, rows that
// fit one stage: each of p.solo warps takes every p.solo-th task by itself, so
// nothing waits for the other warps (a short task's barrier and sum took
// longer than its weights: 16 tokens over 4-bit experts, 83 of them at
// d = 2048, F = 768, ran 261 us that way).  The number of stages (and of scale
// slots) is a multiple of p.solo, so within a part a stage always serves the
// same warp: a barrier's parity tells a warp only whether the use it waits
// for is over if it has seen the one before.
template <int FMT, int PART, int NB, bool SOLO>
__device__ __noinline__ void consume_part(const FewParams &p, Ring &r, uint32_t &red_it) {
  Shared *sh = r.sh;
  constexpr bool PHASE2 = PART == S2 || PART == R2;
  constexpr bool LO = PHASE2 && FMT == BF16;
  constexpr int NBP = FMT == Q4 ? 1 : NB;   // blocks of eight tokens whose operand is fetched ahead
  constexpr int R = ratio_of<FMT>();
  const Dims dm = part_dims(p, PART, sh->nact);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int K = !PHASE2 ? p.d : (PART == S2 ? p.Fs : p.F);
  const int rb = row_bytes<FMT>(K);
  const int groups = K / 64;
  const size_t lo_bytes = 2 * (PART == S2 ? p.hs_lo : p.h_lo);
  const int w0 = SOLO ? 0 : warp * 64;      // this warp's first segment of a piece
  constexpr int STEP = SOLO ? 64 : CW * 64; // and the distance to its next
  constexpr int SEGS = segs_of<FMT>();
  constexpr int FULL = SEGS * STEP;         // bytes of a row in a whole piece
  const int start = min(min(FULL, p.ch), rb);   // and in a row's first
  const int lane_b = (w0 + c * (FMT == Q4 ? 8 : 16)) * R;
  const uint32_t row_lo = g * (p.ch + pad_of(FMT)) + w0 + c * (FMT == Q4 ? 8 : 16);
  const uint32_t row_hi = row_lo + 8 * (p.ch + pad_of(FMT));
  const int mine = dm.n, end = dm.first + dm.n;       // tasks of this block
  if (mine == 0) return;
  const int stride = SOLO ? p.solo : 1;
  uint32_t st = r.st, ph = r.ph, sc_st = r.sc_st, sc_ph = r.sc_ph;
  const int skip = SOLO ? min(warp, mine) : 0;
  for (int i = 0; i < skip; ++i) {
    advance(st, ph, p.stages);
    if (FMT == Q4) advance(sc_st, sc_ph, p.sc_slots);
  }

  Cursor cu;
  cu.task = dm.first + (SOLO ? warp : 0);
  if (cu.task < end && (!SOLO || warp < p.solo)) {
    place<PART>(p, sh, dm, cu);
    const char *bp[NB];                     // the piece's stretch of the token rows, at this lane
    BSeg<FMT, LO> bv[SEGS][NBP];
#pragma unroll
    for (int n = 0; n < NB; ++n) bp[n] = b_row<FMT, PART>(p, cu, g + 8 * n) + lane_b;
#pragma unroll
    for (int s = 0; s < SEGS; ++s)
#pragma unroll
      for (int n = 0; n < NBP; ++n)
        load_b<FMT, LO, true>(bv[s][n], bp[n] + s * STEP * R, lo_bytes, start - w0 - s * STEP, c);

    for (;;) {
      Acc<FMT, NB> acc;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc.f[n][0][j] = acc.f[n][1][j] = 0;
      Cursor nx = cu;
      nx.task += stride;
      const bool more = nx.task < end;
      const bool second = cu.rows > 8;
      const uint16_t *sc = nullptr;
      if (FMT == Q4) {
        wait_on(&sh->sc_full[sc_st], sc_ph, sh, p, kDevTimeoutEpilogue);
        sc = reinterpret_cast<const uint16_t *>(r.sc + (size_t)sc_st * p.sc_slot) + g * groups + w0 / 32;
      }
      int in = 0;                           // bytes of the rows before this piece in its stage
      for (int off = 0, left; off < rb; off += left) {
        left = min(min(FULL, p.ch - in), rb - off);
        // where the next piece's token operand comes from: its loads take the
        // registers of each segment as soon as that has been used
        const bool last = off + left >= rb;
        const bool ends = last || in + left == p.ch;        // of the stage
        const char *bn[NB];
        int next_left;                      // bytes of the weight rows in the next piece, none: 0
        if (!last) {
          next_left = min(min(FULL, ends ? p.ch : p.ch - in - left), rb - off - left);
#pragma unroll
          for (int n = 0; n < NB; ++n) bn[n] = bp[n] + left * R;
        } else {
          next_left = more ? start : 0;
          if (more) place<PART>(p, sh, dm, nx);
#pragma unroll
          for (int n = 0; n < NB; ++n) bn[n] = more ? b_row<FMT, PART>(p, nx, g + 8 * n) + lane_b : bp[n];
        }
        const uint8_t *tile = r.tiles + (size_t)st * p.stage_bytes + in;
        if (in == 0) wait_on(&sh->full[st], ph, sh, p, kDevTimeoutEpilogue);
        __syncwarp();
        if (left == FULL && next_left == FULL) {
#pragma unroll
          for (int s = 0; s < SEGS; ++s) {
            consume<FMT, LO, NB, NBP, false>(acc, bv[s], bp[NB - 1] + s * STEP * R, 64, tile + row_lo + s * STEP,
                                             tile + row_hi + s * STEP, second, c, sc + (off + s * STEP) / 32, groups);
#pragma unroll
            for (int n = 0; n < NBP; ++n) load_b<FMT, LO, false>(bv[s][n], bn[n] + s * STEP * R, lo_bytes, 64, c);
          }
        } else {
#pragma unroll
          for (int s = 0; s < SEGS; ++s) {
            const int at = w0 + s * STEP;
            if (at < left)
              consume<FMT, LO, NB, NBP, true>(acc, bv[s], bp[NB - 1] + s * STEP * R, left - at,
                                              tile + row_lo + s * STEP, tile + row_hi + s * STEP, second, c,
                                              sc + (off + s * STEP) / 32, groups);
#pragma unroll
            for (int n = 0; n < NBP; ++n)
              load_b<FMT, LO, true>(bv[s][n], bn[n] + s * STEP * R, lo_bytes, next_left - at, c);
          }
        }
        if (ends) {
          __syncwarp();
          if (lane == 0) mbar_arrive_n(&sh->empty[st], SOLO ? CW : 1);
          if (!SOLO) advance(st, ph, p.stages);
          in = 0;
        } else {
          in += left;
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) bp[n] = bn[n];
      }
      if (SOLO) {
        if (FMT == Q4 && lane == 0) mbar_arrive(&sh->sc_empty[sc_st]);
        for (int i = 0; i < p.solo; ++i) {
          advance(st, ph, p.stages);
          if (FMT == Q4) advance(sc_st, sc_ph, p.sc_slots);
        }
        // accumulators 0, 1: row g, tokens 2c, 2c + 1; 2, 3: row g + 8
        const bool pairs = PART == S1 || (PART == R1 && p.swiglu);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (n > 0 && !second) break;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int tok = 8 * n + 2 * c + j;
            const float a = (float)(acc.f[n][0][j] + acc.f[n][1][j]);
            const float b = (float)(acc.f[n][0][j + 2] + acc.f[n][1][j + 2]);
            float m = emit<FMT, PART>(p, cu, g, tok, a, b);
            if (!pairs) m = abs_max(m, emit<FMT, PART>(p, cu, g + 8, tok, b, 0.f));
            if (FMT == I8 && PART == R1) {
              uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
              if (g == 0 && tok < cu.rows) atomicMax(p.rowmax + cu.row0 + tok, top);
            }
          }
        }
      } else {
        // the eight warps' partial results meet; two buffers in turn, so one
        // barrier per task keeps writers and readers apart
        uint32_t(*red)[2][32][4] = sh->red[red_it & 1u];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          uint32_t v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const auto sum = acc.f[n][0][j] + acc.f[n][1][j];
            if constexpr (FMT == I8) v[j] = (uint32_t)sum;
            else v[j] = __float_as_uint(sum);
          }
          *reinterpret_cast<uint4 *>(red[warp][n][lane]) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        consumer_sync();
        if (FMT == Q4) {
          if (threadIdx.x == 0) mbar_arrive(&sh->sc_empty[sc_st]);
          advance(sc_st, sc_ph, p.sc_slots);
        }
        ++red_it;
        // value (row, token) of the task: accumulator j of lane 4 (row % 8) + (token % 8) / 2
        auto total = [&](int row, int tok) {
          const int ln = (row & 7) * 4 + ((tok & 7) >> 1), j = (tok & 1) + (row >> 3) * 2, n = tok >> 3;
          if (FMT == I8) {
            int v = 0;
#pragma unroll
            for (int w = 0; w < CW; ++w) v += (int)red[w][n][ln][j];
            return (float)v;
          }
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < CW; ++w) v += __uint_as_float(red[w][n][ln][j]);
          return v;
        };
        const bool pairs = PART == S1 || (PART == R1 && p.swiglu);
        const int cols = pairs ? 8 : ROWS;
        const int most = cols * 8 * (second ? 2 : 1);
        for (int i = threadIdx.x; i < most; i += CT) {            // whole warps take part
          const int tok = i / cols, f = i - tok * cols;
          const float m = tok < cu.rows ? emit<FMT, PART>(p, cu, f, tok, total(f, tok), pairs ? total(f + 8, tok) : 0.f) : 0.f;
          if (FMT == I8 && PART == R1) {
            // the row's largest |h|: over the task's columns (8 or 16 neighbouring lanes), then the grid
            uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;
            for (int o = 1; o < cols; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (f == 0 && tok < cu.rows) atomicMax(p.rowmax + cu.row0 + tok, top);
          }
        }
      }
      if (!more) break;
      cu = nx;
    }
  }
  // every warp leaves the part at the same place of the ring, and together:
  // the next part's uses follow ones that other warps waited for
  if (SOLO) {
    consumer_sync();
    const uint32_t n = r.st + mine;
    r.ph ^= n / p.stages & 1u;
    r.st = n % p.stages;
    if (FMT == Q4) {
      const uint32_t m = r.sc_st + mine;
      r.sc_ph ^= m / p.sc_slots & 1u;
      r.sc_st = m % p.sc_slots;
    }
  } else {
    r.st = st;
    r.ph = ph;
    r.sc_st = sc_st;
    r.sc_ph = sc_ph;
  }
}

template <int FMT, int PART, int NB>
__device__ __forceinline__ void run_part(const FewParams &p, Ring &r, uint32_t &red_it) {
  const int K = PART == S1 || PART == R1 ? p.d : (PART == S2 ? p.Fs : p.F);
  if (row_bytes<FMT>(K) <= p.ch && p.solo >= CW / 2) consume_part<FMT, PART, NB, true>(p, r, red_it);
  else consume_part<FMT, PART, NB, false>(p, r, red_it);
}

// ---------------------------------------------------------------- router
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// The order-preserving 64-bit image of a float64 (-0 as +0, NaN below all),
// and back.  Comparing images costs integer instructions; a float64
// comparison is several times slower here.
__device__ __forceinline__ unsigned long long key_of(double v) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
  return v == v ? ((u >> 63) ? ~u : (u | 0x8000000000000000ull)) : 0ull;
}
__device__ __forceinline__ double of_key(unsigned long long k) {
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7FFFFFFFFFFFFFFFull) : ~k));
}
// Warp arg-max of (key, i), ties to the lower i; returns i
__device__ __forceinline__ int warp_argmax(unsigned long long key, int i) {
  const unsigned full = 0xffffffffu;
  const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
  const bool top = hi == __reduce_max_sync(full, hi);
  const unsigned who = __ballot_sync(full, top);
  if (__popc(who) == 1) return __shfl_sync(full, i, __ffs(who) - 1);
  const uint32_t mlo = __reduce_max_sync(full, top ? lo : 0u);
  return (int)__reduce_min_sync(full, top && lo == mlo ? (uint32_t)i : 0xFFFFFFFFu);
}

// Logits: `per` warps of a block share an expert, each a slice of the hidden
// dimension; their sums meet in shared memory, in slice order.
template <int TP>
__device__ __forceinline__ void route_logits(const FewParams &p, Shared *sh) {
  constexpr int IT = TP <= 4 ? 8 : (TP <= 8 ? 4 : 2);   // steps of 256 elements whose weights are in flight at once
  double(*sums)[MAX_T] = reinterpret_cast<double(*)[MAX_T]>(sh->red);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = p.E <= (int)gridDim.x ? CW : CW / 2, at_once = CW / per;
  const int slice = ((p.d + per - 1) / per + 7) / 8 * 8;
  for (int e0 = blockIdx.x * at_once; e0 < p.E; e0 += gridDim.x * at_once) {
    const int e = e0 + warp / per;
    double acc[TP];
#pragma unroll
    for (int t = 0; t < TP; ++t) acc[t] = 0.0;
    const int k1 = e < p.E ? min(p.d, (warp % per + 1) * slice) : 0;
    const float *w = p.w_router + (size_t)min(e, p.E - 1) * p.d;
#pragma unroll 1
    for (int k0 = (warp % per) * slice; k0 < k1; k0 += 256 * IT) {
      float4 wv[IT][2];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int k = k0 + (lane + 32 * i) * 8;
        wv[i][0] = wv[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < k1) {
          wv[i][0] = __ldg(reinterpret_cast<const float4 *>(w + k));
          wv[i][1] = __ldg(reinterpret_cast<const float4 *>(w + k + 4));
        }
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int k = k0 + (lane + 32 * i) * 8;
        if (k < k1) {
          const float4 wa = wv[i][0], wb = wv[i][1];
#pragma unroll
          for (int t = 0; t < TP; ++t) {
            if (t < p.T) {
              const uint4 xv = __ldg(reinterpret_cast<const uint4 *>(p.x + (size_t)t * p.d + k));
              float run = __uint_as_float(xv.x << 16) * wa.x;
              run = fmaf(__uint_as_float(xv.x & 0xffff0000u), wa.y, run);
              run = fmaf(__uint_as_float(xv.y << 16), wa.z, run);
              run = fmaf(__uint_as_float(xv.y & 0xffff0000u), wa.w, run);
              run = fmaf(__uint_as_float(xv.z << 16), wb.x, run);
              run = fmaf(__uint_as_float(xv.z & 0xffff0000u), wb.y, run);
              run = fmaf(__uint_as_float(xv.w << 16), wb.z, run);
              run = fmaf(__uint_as_float(xv.w & 0xffff0000u), wb.w, run);
              acc[t] += (double)run;
            }
          }
        }
      }
    }
    // halving exchanges: each step keeps half of the tokens' sums on each half of the lanes
    int have = TP;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (have > 1) {
        have >>= 1;
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < TP / 2; ++i)
          if (i < have) {
            const double give = up ? acc[i] : acc[i + have];
            acc[i] = (up ? acc[i + have] : acc[i]) + __shfl_xor_sync(0xffffffffu, give, o);
          }
      } else {
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
      }
    }
    // the lane's token: its bits from 16 down chose the halves
    constexpr int LOG = TP == 16 ? 4 : (TP == 8 ? 3 : (TP == 4 ? 2 : 0));
    if ((lane & ((32 >> LOG) - 1)) == 0) sums[warp][lane >> (5 - LOG)] = acc[0];
    consumer_sync();
    for (int i = threadIdx.x; i < at_once * p.T; i += CT) {
      const int t = i / at_once, q = i - t * at_once;
      double s = 0.0;
      for (int j = 0; j < per; ++j) s += sums[q * per + j][t];
      if (e0 + q < p.E) p.logits[(size_t)t * p.E + e0 + q] = s;
    }
    consumer_sync();
  }
}

constexpr int EPL = kMaxExperts / 32;

// One token's choice from its row of `prob` (softmax: shifted logits, made
// probabilities here; sigmoid: probabilities); ids and weights to shared
// memory.  A warp; expert lane + 32 j.  keys: this warp's scratch.
__device__ __forceinline__ void choose(const FewParams &p, Shared *sh, int t, double *prob, unsigned long long *keys,
                                       int lane) {
  const int E = p.E;
  constexpr unsigned long long LOWEST = 0x000FFFFFFFFFFFFFull;   // key of -infinity
  unsigned long long key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) key[j] = lane + 32 * j < E ? key_of(prob[lane + 32 * j]) : 0ull;
  unsigned long long best = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) best = max(best, key[j]);
  // a token without a single number among its scores chooses nothing
  const bool none = !__any_sync(0xffffffffu, best != 0ull);
  if (p.router == MOE_ROUTER_SOFTMAX_TOPK) {
    const double m = warp_max(best ? of_key(best) : -INFINITY);
    double s = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
      const double v = exp(prob[e] - m);
      prob[e] = v;
      s += v;
    }
    const double inv = 1.0 / warp_sum(s);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 32 * j < E) {
        const double v = prob[lane + 32 * j] * inv;
        prob[lane + 32 * j] = v;
        key[j] = key_of(v);
      }
    __syncwarp();
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (e < E) {
        if (p.bias) key[j] = key_of(prob[e] + (double)__ldg(p.bias + e));
        keys[e] = key[j];
      }
    }
    __syncwarp();
    // group score = sum of the two largest selection scores in the group
    const int G = E / p.n_group;
    unsigned long long gkey = 0;
    if (lane < p.n_group) {
      unsigned long long b1 = 0, b2 = 0;
#pragma unroll 4
      for (int q = 0; q < G; ++q) {
        const unsigned long long v = keys[lane * G + q];
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
      gkey = key_of((b1 ? of_key(b1) : -INFINITY) + (b2 ? of_key(b2) : -INFINITY));
    }
    uint32_t keep = 0;
#pragma unroll 1
    for (int r = 0; r < p.topk_group; ++r) {
      const bool open = lane < p.n_group && !((keep >> lane) & 1u);
      const int gi = warp_argmax(open ? gkey : 0ull, open ? lane : 0x7fffffff);
      keep |= 1u << (gi & 31);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (e < E && !((keep >> (e / G)) & 1u)) key[j] = min(key[j], LOWEST);
    }
  }

  int my_e = 0x7fffffff;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    unsigned long long bk = 0;
    int bi = 0x7fffffff;
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j)                 // ties: the lower expert
      if (key[j] >= bk && key[j] != 0ull) {
        bk = key[j];
        bi = lane + 32 * j;
      }
    bi = warp_argmax(bk, bi);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (bi == lane + 32 * j) key[j] = 0ull;          // taken
    if (lane == r) my_e = bi;
  }
  const bool bad = none || my_e < 0 || my_e >= E;
  const double my_w = lane < p.k && !bad ? prob[my_e] : 0.0;
  const double tot = warp_sum(my_w);
  double wout;
  if (p.router == MOE_ROUTER_SOFTMAX_TOPK) wout = p.norm ? my_w / fmax(tot, 1e-12) : my_w;
  else wout = (p.norm ? my_w / (tot + 1e-20) : my_w) * p.scaling;
  if (lane < p.k) {
    if (bad && blockIdx.x == 0) record_status(p.status, kDevBadExpertId);
    sh->sel_id[t * p.k + lane] = bad ? -1 : my_e;
    sh->sel_w[t * p.k + lane] = (float)wout;
  }
}

// Choice for every token and the plan, the same in every block.  The loops
// that run once per expert stay rolled: a block runs this code once per
// launch, and fetching its instructions is much of its time.
__device__ __noinline__ void make_plan(const FewParams &p, Shared *sh, double *prob) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(sizeof(((Shared *)0)->red) >= CW * kMaxExperts * 8, "selection scratch");
  unsigned long long *keys = reinterpret_cast<unsigned long long *>(sh->red) + warp * kMaxExperts;
  sh->mask[tid] = 0u;
  static_assert(CT == kMaxExperts, "a thread per expert");
  // logits (softmax: with the bias) or sigmoid scores, a thread per (token, expert)
  const int n_logits = p.T * p.E;
#pragma unroll 1
  for (int i0 = tid; i0 < n_logits; i0 += 8 * CT) {    // eight loads in flight at a time
    double v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + u * CT < n_logits ? __ldcg(p.logits + i0 + u * CT) : 0.0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * CT < n_logits) prob[i0 + u * CT] = v[u];
  }
#pragma unroll 1
  for (int i = tid; i < p.T * p.E; i += CT) {
    double l = prob[i];
    if (p.router == MOE_ROUTER_SOFTMAX_TOPK) {
      if (p.bias) l += (double)__ldg(p.bias + i % p.E);
    } else {
      l = 1.0 / (1.0 + exp(-l));
    }
    prob[i] = l;
  }
  consumer_sync();
#pragma unroll 1
  for (int t = warp; t < p.T; t += CW) choose(p, sh, t, prob + (size_t)t * p.E, keys, lane);
  consumer_sync();
  const int slots = p.T * p.k;
#pragma unroll 1
  for (int i = tid; i < slots; i += CT) {
    const int e = sh->sel_id[i];
    if (e >= 0) atomicOr(&sh->mask[e], 1u << (i / p.k));
  }
  consumer_sync();
  // thread e: expert e.  In-order dropping: the first `cap` tokens stay
  uint32_t m = sh->mask[tid];
  const int raw = __popc(m);
  if (p.cap >= 0)
    while (__popc(m) > p.cap) m &= ~(0x80000000u >> __clz(m));
  const int cnt = __popc(m);
  const unsigned live = __ballot_sync(0xffffffffu, cnt > 0);
  int pre = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) {
    sh->warp_n[warp] = __popc(live);
    sh->warp_rows[warp] = pre;
  }
  sh->mask[tid] = m;
  consumer_sync();
  int n = 0, rows = 0, all_n = 0, all_rows = 0;
#pragma unroll
  for (int w = 0; w < CW; ++w) {
    if (w == warp) {
      n = all_n;
      rows = all_rows;
    }
    all_n += sh->warp_n[w];
    all_rows += sh->warp_rows[w];
  }
  if (cnt > 0) {
    const int at = n + __popc(live & ((1u << lane) - 1u));
    sh->act[at] = (int16_t)tid;
    sh->row0[at] = (int16_t)(rows + pre - cnt);
  }
  if (tid == 0) {
    sh->nact = all_n;
    sh->row0[all_n] = (int16_t)all_rows;
  }
  consumer_sync();
  if (tid == 0) mbar_arrive(&sh->plan);
  if (blockIdx.x == 0) {
    for (int i = tid; i < slots; i += CT) {
      p.ids[i] = sh->sel_id[i];
      p.wts[i] = sh->sel_w[i];
    }
    if (tid < p.E) {
      double s = 0.0;
      for (int t = 0; t < p.T; ++t) s += prob[(size_t)t * p.E + tid];
      p.prob_sum[tid] = (float)s;
      p.raw_counts[tid] = raw;
      p.kept_counts[tid] = cnt;
      if (raw > cnt) atomicAdd(p.dropped, raw - cnt);
    }
  }
}

// Row of every slot, for the combine
__device__ __forceinline__ void slot_rows(const FewParams &p, Shared *sh) {
  for (int i = threadIdx.x; i < p.T * p.k; i += CT) {
    const int e = sh->sel_id[i], t = i / p.k;
    int row = -1;
    if (e >= 0 && (sh->mask[e] >> t & 1u)) {
      int lo = 0, hi = sh->nact;            // act is ascending
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sh->act[mid] <= e) lo = mid; else hi = mid;
      }
      row = sh->row0[lo] + __popc(sh->mask[e] & ((1u << t) - 1u));
    }
    sh->slot_row[i] = (int16_t)row;
  }
}

// ---------------------------------------------------------------- 8-bit codes
__device__ __forceinline__ uint32_t abs_max2(uint32_t w, uint32_t m) {
  return max(m, max((w << 16) & 0x7FFF0000u, w & 0x7FFF0000u));
}

// Codes of 8 bf16 elements of a row with largest magnitude `top` (fp32 bits):
// rne(127 x / a), see the row quantisation kernel for why this is exact.
__device__ __forceinline__ uint2 codes8(uint4 v, uint32_t top) {
  if (top == 0u || top >= 0x7F800000u) return make_uint2(0u, 0u);
  float a = __uint_as_float(top);
  const float pre = a < 0x1p-60f ? 0x1p64f : (a > 0x1p100f ? 0x1p-32f : 1.f);
  a *= pre;
  const float r = __frcp_rn(a);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    const float t = 127.f * (x * pre), p0 = t * r;
    q[i] = __float_as_uint(__fmaf_rn(__fmaf_rn(-p0, a, t), r, p0) + 12582912.f);
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
  return o;
}

// token rows: one block each, from the last block down (the router's units
// start at the first)
__device__ __forceinline__ void quantize_x(const FewParams &p, Shared *sh) {
  uint32_t *scratch = &sh->red[0][0][0][0][0];
  for (int t = (int)gridDim.x - 1 - (int)blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4 *row = reinterpret_cast<const uint4 *>(p.x + (size_t)t * p.d);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.d / 8; i += CT) {
      const uint4 v = __ldg(row + i);
      m = abs_max2(v.x, abs_max2(v.y, abs_max2(v.z, abs_max2(v.w, m))));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    consumer_sync();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = m;
    consumer_sync();
    for (int w = 0; w < CW; ++w) m = max(m, scratch[w]);
    for (int i = threadIdx.x; i < p.d / 8; i += CT)
      reinterpret_cast<uint2 *>(p.xq + (size_t)t * p.d)[i] = codes8(__ldg(row + i), m);
    if (threadIdx.x == 0)
      p.xs[t] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(m), 127.f);
    consumer_sync();                        // the scratch has been read
  }
}

// rows of h, all blocks together
__device__ __forceinline__ void quantize_h(const FewParams &p, const Shared *sh) {
  const int rows = sh->row0[sh->nact], nv = p.F / 8;
  for (long long i = (long long)blockIdx.x * CT + threadIdx.x; i < (long long)rows * nv; i += (long long)gridDim.x * CT) {
    const int r = (int)(i / nv);
    reinterpret_cast<uint2 *>(p.hq)[i] =
        codes8(__ldcg(reinterpret_cast<const uint4 *>(p.h) + i), __ldcg(p.rowmax + r));
  }
}

// out[t] = sum_j w_j y[slot_row] in slot order (+ the shared expert's row), 4 columns per thread
__device__ __forceinline__ void combine(const FewParams &p, const Shared *sh) {
  const int nv = p.d / 4;
  for (int i = blockIdx.x * CT + threadIdx.x; i < p.T * nv; i += gridDim.x * CT) {
    const int t = i / nv, c = i - t * nv;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.k; ++j) {
      const int row = sh->slot_row[t * p.k + j];
      if (row < 0) continue;
      const float w = sh->sel_w[t * p.k + j];
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)row * p.d) + c);
      a[0] = fmaf(w, v.x, a[0]);
      a[1] = fmaf(w, v.y, a[1]);
      a[2] = fmaf(w, v.z, a[2]);
      a[3] = fmaf(w, v.w, a[3]);
    }
    if (p.Fs) {
      const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.y + (size_t)(p.T * p.k + t) * p.d) + c);
      a[0] += v.x;
      a[1] += v.y;
      a[2] += v.z;
      a[3] += v.w;
    }
    *reinterpret_cast<uint2 *>(p.out + (size_t)t * p.d + 4 * c) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
  }
}

template <int FMT, int TP>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ FewParams p) {
  constexpr int NB = TP > 8 ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Ring r;
  r.tiles = smem_raw;
  r.sc = smem_raw + (size_t)p.stages * p.stage_bytes;
  r.scratch = r.sc + (size_t)p.sc_slots * p.sc_slot;
  r.sh = reinterpret_cast<Shared *>(r.scratch + scratch_bytes(p.T, p.E));
  r.st = r.ph = r.sc_st = r.sc_ph = r.issued = r.sc_issued = 0;
  r.ok = true;
  Shared *sh = r.sh;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], CW);
    }
    for (int s = 0; s < MAX_SC; ++s) {
      mbar_init(&sh->sc_full[s], 1);
      mbar_init(&sh->sc_empty[s], 1);
    }
    mbar_init(&sh->plan, 1);
    sh->abort_flag = 0;
    sh->nact = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncthreads();
  volatile int *abort_flag = &sh->abort_flag;

  if (warp == CW) {
    if (p.Fs) produce_part<BF16>(p, r, S1, 0);
    if (p.Fs && r.ok) produce_part<BF16>(p, r, S2, 0);
    if (r.ok)
      r.ok = wait_bounded(&sh->plan, 0u, abort_flag, p.status, kDevTimeoutProducer, p.timeout_ns);
    r.ok = __all_sync(0xffffffffu, r.ok);
    const int nact = r.ok ? sh->nact : 0;
    if (r.ok) produce_part<FMT>(p, r, R1, nact);
    if (r.ok) produce_part<FMT>(p, r, R2, nact);
    if ((threadIdx.x & 31) == 0 && !r.ok) {
      // copies already issued land before the block goes away
      const uint32_t n = p.stages, m = p.sc_slots;
      for (uint32_t i = r.issued > n ? r.issued - n : 0u; i < r.issued; ++i)
        if (!wait_drain(&sh->full[i % n], (i / n) & 1u)) record_status(p.status, kDevTimeoutDrain);
      for (uint32_t i = r.sc_issued > m ? r.sc_issued - m : 0u; i < r.sc_issued; ++i)
        if (!wait_drain(&sh->sc_full[i % m], (i / m) & 1u)) record_status(p.status, kDevTimeoutDrain);
    }
  } else {
    uint32_t red_it = 0;
    if (FMT == I8) {
      quantize_x(p, sh);
      if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.T * p.k; i += CT) p.rowmax[i] = 0u;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.dropped = 0;
    route_logits<TP>(p, sh);
    if (p.Fs) run_part<BF16, S1, NB>(p, r, red_it);
    grid_arrive(p.bar);
    grid_wait(p.bar, abort_flag, p);
    make_plan(p, sh, reinterpret_cast<double *>(r.scratch));
    if (p.Fs) run_part<BF16, S2, NB>(p, r, red_it);
    run_part<FMT, R1, NB>(p, r, red_it);
    grid_arrive(p.bar + 8);
    grid_wait(p.bar + 8, abort_flag, p);
    if (FMT == I8) {
      quantize_h(p, sh);
      grid_arrive(p.bar + 16);
      grid_wait(p.bar + 16, abort_flag, p);
    }
    run_part<FMT, R2, NB>(p, r, red_it);
    grid_arrive(p.bar + 24);
    slot_rows(p, sh);
    grid_wait(p.bar + 24, abort_flag, p);
    combine(p, sh);
  }
  __syncthreads();
}

template <int FMT, int TP>
cudaError_t run(FewParams &p, cudaStream_t s) {
  const size_t fixed = sizeof(Shared) + scratch_bytes(p.T, p.E) + (size_t)p.sc_slots * p.sc_slot;
  int stages = (int)((SMEM_LIMIT - fixed) / p.stage_bytes);
  stages = stages < MAX_STAGES ? stages : MAX_STAGES;
  p.solo = p.sc_slots && p.sc_slots < CW ? p.sc_slots : CW;
  p.solo = stages < p.solo ? stages : p.solo;
  if (p.sc_slots) p.sc_slots -= p.sc_slots % p.solo;
  p.stages = stages - stages % p.solo;
  const size_t smem = fixed + (size_t)p.stages * p.stage_bytes;
  auto kern = few_kernel<FMT, TP>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  note_launch();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;      // the blocks wait for one another
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = sm_count();
  cfg.blockDim = THREADS;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int FMT>
cudaError_t run_t(FewParams &p, cudaStream_t s) {
  if (p.T <= 1) return run<FMT, 1>(p, s);
  if (p.T <= 4) return run<FMT, 4>(p, s);
  if (p.T <= 8) return run<FMT, 8>(p, s);
  return run<FMT, 16>(p, s);
}

struct FewLayout {
  size_t logits, xq, xs, h, h_lo, hs, hs_lo, rowmax, hq, y, total;
};

FewLayout few_layout(const moe_config &c) {
  FewLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t here = off;
    off = align_up(off + bytes, 256);
    return here;
  };
  const size_t T = c.num_tokens, S = T * c.top_k, d = c.hidden, F = c.intermediate;
  const size_t Fs = c.shared_intermediate > 0 ? c.shared_intermediate : 0;
  const bool i8 = c.weight_dtype == MOE_I8_CHANNEL;
  L.logits = take(sizeof(double) * T * c.num_experts);
  L.xq = take(i8 ? T * d : 0);
  L.xs = take(i8 ? sizeof(float) * T : 0);
  L.h = take(2 * S * F);
  L.h_lo = take(i8 ? 0 : 2 * S * F);
  L.hs = take(2 * T * Fs);
  L.hs_lo = take(2 * T * Fs);
  L.rowmax = take(i8 ? sizeof(unsigned) * S : 0);
  L.hq = take(i8 ? S * F : 0);
  L.y = take(sizeof(float) * (S + (Fs ? T : 0)) * d);
  L.total = off;
  return L;
}

// bytes of a row per stage: the longest row if that is short, so that short
// rows get more stages
int stage_ch(const moe_config &c) {
  const long long K = c.hidden > c.intermediate ? c.hidden : c.intermediate;
  long long b = c.weight_dtype == MOE_BF16 ? 2 * K : (c.weight_dtype == MOE_I8_CHANNEL ? K : K / 2);
  if (c.shared_intermediate > 0) {
    const long long s = 2LL * (c.hidden > c.shared_intermediate ? c.hidden : c.shared_intermediate);
    b = b > s ? b : s;
  }
  b = (b + 127) / 128 * 128;
  return (int)(b < MAX_CH ? b : MAX_CH);
}

int scale_slot(const moe_config &c) {
  // 16 rows of K/64 scales and biases, 2 bytes each
  const int K = c.hidden > c.intermediate ? c.hidden : c.intermediate;
  return c.weight_dtype == MOE_Q4_AFFINE_G64 ? K / 64 * 2 * 2 * ROWS : 0;
}

int scale_slots(const moe_config &c) {
  const int b = scale_slot(c);
  const int n = b ? SC_BYTES / b : 0;
  return b == 0 ? 0 : (n < 2 ? 2 : (n > MAX_SC ? MAX_SC : n));
}

}  // namespace

bool few_supported(const moe_config &c) {
  if (c.num_tokens > kFewTokens || c.act_dtype != MOE_BF16) return false;
  // at least three stages beside the scales
  return sizeof(Shared) + scratch_bytes(c.num_tokens, c.num_experts) + (size_t)scale_slots(c) * scale_slot(c) + 3 * (size_t)(ROWS * (MAX_CH + 64)) <= (size_t)SMEM_LIMIT;
}

size_t few_bytes(const moe_config &c) { return few_supported(c) ? few_layout(c).total : 0; }

cudaError_t launch_few(const FewArgs &a, cudaStream_t s) {
  const moe_config &c = *a.cfg;
  const FewLayout L = few_layout(c);
  FewParams p{};
  p.timeout_ns = wait_timeout_ns();
  p.T = c.num_tokens;
  p.d = c.hidden;
  p.F = c.intermediate;
  p.E = c.num_experts;
  p.k = c.top_k;
  p.Fs = c.shared_intermediate > 0 ? c.shared_intermediate : 0;
  p.router = c.router;
  p.norm = c.norm_topk_prob;
  p.scaling = (double)c.routed_scaling;
  p.n_group = c.n_group;
  p.topk_group = c.topk_group;
  p.cap = a.capacity < 0 || a.capacity > kFewTokens ? -1 : (int)a.capacity;
  p.swiglu = c.act == MOE_ACT_SWIGLU;
  p.x = static_cast<const uint16_t *>(a.x);
  p.w_router = a.w_router;
  p.bias = a.router_bias;
  p.w1 = a.w1; p.w2 = a.w2; p.w3 = a.w3;
  p.s1 = a.s1; p.s2 = a.s2; p.s3 = a.s3;
  p.b1 = a.b1; p.b2 = a.b2; p.b3 = a.b3;
  p.w_stride = a.w_stride;
  p.sw1 = static_cast<const uint16_t *>(a.shared_w1);
  p.sw2 = static_cast<const uint16_t *>(a.shared_w2);
  p.sw3 = static_cast<const uint16_t *>(a.shared_w3);
  p.out = static_cast<uint16_t *>(a.out);
  p.ids = a.ids;
  p.wts = a.wts;
  p.raw_counts = a.raw_counts;
  p.kept_counts = a.kept_counts;
  p.dropped = a.dropped;
  p.prob_sum = a.prob_sum;
  p.status = a.status;
  p.bar = reinterpret_cast<unsigned *>(a.status) + 16;
  char *ws = static_cast<char *>(a.ws);
  p.logits = reinterpret_cast<double *>(ws + L.logits);
  p.xq = reinterpret_cast<int8_t *>(ws + L.xq);
  p.xs = reinterpret_cast<float *>(ws + L.xs);
  p.h = reinterpret_cast<uint16_t *>(ws + L.h);
  p.h_lo = (L.h_lo - L.h) / 2;
  p.hs = reinterpret_cast<uint16_t *>(ws + L.hs);
  p.hs_lo = (L.hs_lo - L.hs) / 2;
  p.rowmax = reinterpret_cast<unsigned *>(ws + L.rowmax);
  p.hq = reinterpret_cast<int8_t *>(ws + L.hq);
  p.y = reinterpret_cast<float *>(ws + L.y);
  p.ch = stage_ch(c);
  p.stage_bytes = ROWS * (p.ch + 64);
  p.sc_slot = scale_slot(c);
  p.sc_slots = scale_slots(c);
  switch (c.weight_dtype) {
    case MOE_BF16: return run_t<BF16>(p, s);
    case MOE_I8_CHANNEL: return run_t<I8>(p, s);
    default: return run_t<Q4>(p, s);
  }
}

}  // namespace moe
