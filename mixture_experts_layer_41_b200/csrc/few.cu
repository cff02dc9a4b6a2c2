// The whole layer for a few tokens (at most 16) in one cooperative kernel.
//
// Between two sampled tokens a server runs the layer on a handful of rows:
// nearly all of its time is reading the chosen experts' weights once.  The
// staged layer spends 9-10 launches on it and gives each weight tile a
// 128-row operand; here one persistent block per SM streams weight rows
// through shared memory from the first product to the last.
//
//   router    the warps of a block share an expert, each a slice of the hidden
//             dimension, times every token (fp32 products over runs of 8,
//             float64 sums);
//   choice    after a grid barrier every block selects for all tokens from
//             the same logits (float64, ties to the lower expert) and builds
//             the same plan: per expert a 16-bit mask of its tokens in token
//             order, cut to the capacity;
//   phase 1   tasks of 16 weight rows: 8 gate rows and the 8 up rows of the
//             same features (ReLU: 16 rows), times the expert's tokens;
//   phase 2   tasks of 16 rows of the down projection, times h;
//   combine   after a last grid barrier: out = sum_j w_j y_j (+ shared).
// The shared expert needs no choice: its phase 1 runs beside the router, its
// phase 2 before the routed experts'.
//
// How the weights move.  Each of a block's sixteen warps walks its own units, 16
// rows x 256 bytes, and each lane fetches with cp.async the 16-byte pieces
// that it will multiply itself, DEPTH units ahead, into slots of its own: there
// is nobody to hand over to, so the stream has no barriers, and it runs on
// across tasks, phases and grid barriers (the slots are full of the next
// phase's weights when a barrier opens).  Measured on 466 MB of 16-row tasks:
// 6.49 TB/s four units deep; one bulk copy per row piece, with a producer
// warp, cost 55 ns each whatever its size (5.1 TB/s at 2 KB, 1.3 at 512 B).
// A block's sixteen warps are two groups of eight, or sixteen on their own; each
// takes a run of consecutive tasks, so most are one expert's and its tokens'
// rows stay in L1.
//
// The product.  mma.sync m16n8: 16 weight rows times 8 tokens.  A thread's
// 16 bytes of rows g and g + 8 and of token g's row are one A and one B
// operand for a permuted order of K (a sum over K has no order), so nothing is
// transposed or shuffled.  At 23 bytes of weights per clock and SM the legacy
// unit (2 clocks a product) is mostly idle.
//   long rows   the eight warps of a group split a task's K; their partial
//               16 x 8 results meet in shared memory, one barrier per task;
//   short rows  (solo) each warp takes whole tasks.
//
// Precision: bf16 weights take h as the sum of two bf16 (16 bits).  8-bit
// weights follow the 8-bit layer's definition (rows of x and of the bf16 h
// quantised).  4-bit weights are bound by unpacking, and integers unpack
// cheapest: a word's eight codes are two registers of four bytes (three
// instructions; as bf16 pairs seven).  So x, and the fp32 h, become integers
// of 16 bits over their row's largest element (an error of 2^-17 of it, far
// below the codes' own), in two digits of 8 bits: v = 256 hi + lo.  Per group
// of 64, s sum(q v) + b sum(v), the sums exact in int32, scaled and added in
// fp32.  Expert outputs stay fp32 until the combine.
//
// Measured (graph replays): one token of d 4096, F 14336, top 2 of 8 in bf16
// 141 us (5.0 TB/s of the weights; the nine launches of the staged layer 306);
// four of d 7168, F 2048, top 8 of 256 in 8 bits with a bf16 shared expert
// 287 us (5.0 TB/s; staged 378); two of d 448, F 256 37 us, all of it launch,
// barriers and latency (16 of them 51, staged 43).  4-bit experts are bound by
// the unpacking and by how evenly few tasks divide: one token of d 2048, F 768,
// top 8 of 128 42 us (staged 53), four 71 (staged 71), 16 tokens 150 us
// (staged 112, with weights rounded to bf16).
//
// Results do not depend on timing: every sum has a fixed order, and the row
// maxima behind the 8-bit codes of h are integer maxima.
// The only waits are the grid barriers, bounded by moe_set_wait_timeout_ns: one
// that runs out records a status and turns every later wait of its block into
// a no-op, so the block runs through its (in-bounds) work and ends.
#include "tc_ptx.cuh"

#include <math.h>

#include <type_traits>

namespace moe {
namespace {

using namespace ptx;

constexpr int CW = 16;                      // warps
constexpr int GW = 8;                       // warps that share a task of long rows: the block has two such groups
constexpr int CT = 32 * CW;
constexpr int ROWS = 16;                    // weight rows per task
constexpr int UNIT = 256;                   // bytes of a row per unit
constexpr int SEG = 64;                     // and per product step: 16 bytes for each lane of a quad
constexpr int SEGS = UNIT / SEG;
constexpr int SOLO_BYTES = 2048;            // rows of at most that many bytes go one task to a warp
constexpr int MAX_KSPLIT = 4;               // parts of K a down-projection task may be cut into
constexpr int MAX_T = kFewTokens;
constexpr int MAX_SLOTS = MAX_T * kMaxTopK;
constexpr int SMEM_LIMIT = 227 * 1024;

enum Fmt { BF16 = 0, I8 = 1, Q4 = 2 };

// units in flight per warp
__host__ __device__ constexpr int depth_of(int fmt, int TP) { return fmt != 2 && TP <= 8 ? 3 : 2; }
// shared memory of one unit: the lanes' pieces, and 32 bytes of scales and biases per lane
__host__ __device__ constexpr int unit_bytes(int fmt) { return ROWS * UNIT + (fmt == Q4 ? 32 * 32 : 0); }

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
  int8_t *xq;                               // 8-bit: [T][d] codes of x; 4-bit: [T][2][d] its two digits
  float *xs;                                // [T] their scales
  float *xg;                                // 4-bit: [T][d/64] sums of x's integers over the groups
  uint16_t *h;                              // [T*k][F], bf16: the low parts h_lo elements further
  float *hf;                                // 4-bit: [T*k][F] in fp32 instead
  size_t h_lo;
  uint16_t *hs;                             // [T][Fs] of the shared expert, likewise
  size_t hs_lo;
  unsigned *rowmax;                         // 8-bit, 4-bit: [T*k] largest |h| of a row, as fp32 bits
  int8_t *hq;                               // 8-bit: [T*k][F] codes; 4-bit: [T*k][2][F] digits
  float *hg;                                // 4-bit: [T*k][F/64]
  float *y;                                 // [ksplit][T*k][d] expert outputs, then [T][d] of the shared expert
  int y_rows;                               // T*k
  int ksplit;                               // most parts of K that y has room for
};

struct Geo {
  int nb;        // row blocks per expert and part of K
  int first, n;  // this block's tasks: first .. first + n - 1
  int rb, ns;    // bytes of a weight row, and its segments
  int ks;        // parts of K
  bool solo;     // one task to a warp
};

// Where a warp's stream stands, as far as it changes from run to run only
struct FeedState {
  Geo g;
  int part, limit;                          // part fetched from, and the first that is not known yet
  int j, run;                               // first task of the run (from the block's first), and its tasks
};

struct __align__(16) Shared {
  FeedState feed[CW];
  int abort_flag;
  int nact;                                 // experts with rows
  uint32_t mask[kMaxExperts];               // tokens an expert keeps
  int16_t act[kMaxExperts];                 // the experts with rows
  int16_t row0[kMaxExperts + 1];            // first row of active expert i
  int sel_id[MAX_SLOTS];
  float sel_w[MAX_SLOTS];
  int16_t slot_row[MAX_SLOTS];
  float bias[kMaxExperts];                  // the router's, zeros without one
  uint8_t raw[kMaxExperts];                 // tokens that chose an expert
  int warp_n[CW], warp_rows[CW];            // per 32 experts: how many have rows, and the rows
};
// Behind it: partial results of the warps, two tasks in turn; scratch of the
// router, and the tokens' probabilities [T][E] while the choice is made
template <int NB>
struct Partial {
  __align__(16) uint32_t red[2][CW][NB][32][4];
};
__device__ __forceinline__ uint32_t *partials(const Shared *sh) {
  return reinterpret_cast<uint32_t *>(const_cast<Shared *>(sh) + 1);
}

// ---------------------------------------------------------------- grid barrier
// Arrival and wait are apart, so work that does not depend on the other blocks
// can run between them.  Both are called by all threads.
__device__ __forceinline__ void grid_arrive(unsigned *ctr) {
  __syncthreads();
  if (threadIdx.x == 0) {
    // (the release covers what the other threads wrote before the barrier above)
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
        record_status(p.status, kDevTimeoutGrid);
        break;
      }
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- tasks
// One task: 16 weight rows.  A block's tasks come in this order: shared phase
// 1, shared phase 2, routed phase 1, routed phase 2; of each part a block
// takes a run of consecutive ones, and the blocks with one task more are
// others from part to part.
enum Part { S1 = 0, S2 = 1, R1 = 2, R2 = 3, END = 4 };

template <int FMT>
__device__ __forceinline__ int row_bytes(int K) {
  return FMT == BF16 ? 2 * K : (FMT == I8 ? K : K / 2);
}

// Tasks of the routed down projection are cut along K while a block has few
// of them: 512 tasks of 28 KB rows on 148 blocks are three or four each, and
// the blocks with three would wait for the others for a quarter of the phase.
__device__ __forceinline__ int k_parts(const FewParams &p, int nact, int rb) {
  int ks = 1;
  while (2 * ks <= p.ksplit && rb >= 2 * SOLO_BYTES * 2 * ks &&
         (long long)nact * ((p.d + ROWS - 1) / ROWS) * ks < 10LL * (int)gridDim.x)
    ks *= 2;
  return ks;
}

template <int FMT>
__device__ __forceinline__ Geo part_geo(const FewParams &p, int part, int nact) {
  const int nbs1 = p.Fs / 8, nbs2 = p.Fs ? (p.d + ROWS - 1) / ROWS : 0;
  const int nb1 = p.swiglu ? p.F / 8 : (p.F + ROWS - 1) / ROWS, nb2 = (p.d + ROWS - 1) / ROWS;
  Geo r;
  r.rb = row_bytes<FMT>(part == S1 || part == R1 ? p.d : (part == S2 ? p.Fs : p.F));
  r.ns = (r.rb + SEG - 1) / SEG;
  r.ks = part == R2 ? k_parts(p, nact, r.rb) : 1;
  r.solo = r.rb <= SOLO_BYTES;
  r.nb = part == S1 ? nbs1 : (part == S2 ? nbs2 : (part == R1 ? nb1 : nb2));
  const int counts[4] = {nbs1, nbs2, nact * nb1, nact * nb2 * r.ks};
  const int G = (int)gridDim.x;
  int skip = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < part) skip += counts[i] % G;
  const int count = part == S1 ? counts[0] : (part == S2 ? counts[1] : (part == R1 ? counts[2] : counts[3]));
  const int b = ((int)blockIdx.x - skip % G + G) % G;
  const int q = count / G, rest = count % G;
  r.n = q + (b < rest ? 1 : 0);
  r.first = b * q + min(b, rest);
  return r;
}

// A task in full: row block b of active expert i, part kp of K
struct Task {
  int i, kp, b;
};
__device__ __forceinline__ Task task_of(const Geo &g, int task) {
  Task t;
  const int blocks = g.nb * g.ks;
  t.i = task / blocks;
  const int w = task - t.i * blocks;
  t.kp = w / g.nb;
  t.b = w - t.kp * g.nb;
  return t;
}

// Segments of the row that this warp takes of a task
struct Span {
  int first, n;
};
__device__ __forceinline__ Span warp_span(const Geo &g, int kp, int warp) {
  const int a = g.ks == 1 ? 0 : kp * g.ns / g.ks, b = g.ks == 1 ? g.ns : (kp + 1) * g.ns / g.ks;
  if (g.solo) return {a, b - a};
  const int w = warp % GW, c = a + w * (b - a) / GW;
  return {c, a + (w + 1) * (b - a) / GW - c};
}

// A warp's (solo) or group's tasks: every `stride`-th of the block's
__device__ __forceinline__ int first_task(const Geo &g, int warp) { return g.solo ? warp : warp / GW; }
__device__ __forceinline__ int task_stride(const Geo &g) { return g.solo ? CW : CW / GW; }
// How many of them, from task j with row block b on, are the same expert's (and part of K's)
__device__ __forceinline__ int run_of(const Geo &g, int j, int b) {
  const int by = task_stride(g);
  return min((g.nb - b + by - 1) / by, (g.n - j + by - 1) / by);
}

// Weight rows of a task: rows 0-7 from w0, 8-15 from w1
struct Src {
  const char *w0, *w1;
  int n0, n1;                               // valid rows of each half
  size_t r0, r1;                            // row index of each half's first (channel scales)
};

__device__ __forceinline__ Src task_src(const FewParams &p, int part, int e, int b, int rb) {
  Src s;
  if (part == S1 || part == R1) {
    const size_t base = part == S1 ? 0 : (size_t)e * p.w_stride;
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

// ---------------------------------------------------------------- the weight stream
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t ld_stream(const void *p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_l1_f32(const float *p) {
  float v;
  asm volatile("ld.global.ca.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ void st_shared4(uint32_t dst, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The fetching end of a warp's stream: the next unit to fetch, DEPTH units
// before the one in use.  Every fetch, and every step at which there is
// nothing to fetch yet, closes a cp.async group, so the unit in use is always
// at least DEPTH groups old.  What changes with tasks only lies in shared
// memory (FeedState); the rest is a lane's own.
struct Feed {
  const char *lo, *hi;                      // this lane's place in rows g and g + 8
  ptrdiff_t step;                           // from a task's end to the next one's begin, within a run
  size_t sc_lo, sc_hi;                      // 4-bit: byte of its scale words of the two rows
  int sc_step;
  int left, nu;                             // units of the task not yet fetched (0: nothing to fetch), and in all
  int run;                                  // tasks of the run, this one included
  int flags;                                // see below; and from bit 8 on the segments of the last unit (0: whole)
  int groups;                               // 4-bit: groups of the row from the next unit's place on
  uint32_t issued, used;                    // units so far
};
// 4-bit: the last unit's scale words, put into its slot a step later
// (four-byte copies straight into shared memory go through L1 and would drive
// the tokens' rows out of it)
struct Words {
  uint32_t w[2][4], at;                     // at 0: none
};
enum FeedFlags { FULL = 1, HAS_LO = 2, HAS_HI = 4, SHORT = 8, DOWN = 16, ODD = 32 };
// FULL: 16 rows of whole segments; HAS_LO / HAS_HI: there is such a row;
// SHORT: the row's last segment, in the task's last unit, ends before this
// lane's piece; DOWN: of the down projection; ODD: 4-bit, the lane's rows begin
// in the middle of a word of scales

// The run that begins with task st.j
template <int FMT>
__device__ __forceinline__ void feed_run(const FewParams &p, const Shared *sh, FeedState &st, Feed &f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const Geo &ge = st.g;
  const Task t = task_of(ge, ge.first + st.j);
  const Span w = warp_span(ge, t.kp, warp);
  const Src s = task_src(p, st.part, st.part >= R1 ? sh->act[t.i] : 0, t.b, ge.rb);
  st.run = run_of(ge, st.j, t.b);
  // a last row block of fewer than 16 rows is a run of its own
  const bool pairs = st.part == S1 || (st.part == R1 && p.swiglu);
  const int N = st.part == S1 ? p.Fs : (st.part == R1 ? p.F : p.d);
  if (!pairs && N % ROWS && st.run > 1 && t.b + (st.run - 1) * task_stride(ge) == ge.nb - 1) --st.run;
  f.run = st.run;
  f.left = f.nu = (w.n + SEGS - 1) / SEGS;
  const bool ends = w.first + w.n == ge.ns;                 // the span reaches the row's end
  const int tail = ge.rb - (ge.ns - 1) * SEG - c * 16;      // of the row from this lane's piece of its last segment on
  f.flags = (ge.rb % SEG == 0 && s.n0 == 8 && s.n1 == 8 ? FULL : 0) | (g < s.n0 ? HAS_LO : 0) |
            (g < s.n1 ? HAS_HI : 0) | (ends && tail <= 0 ? SHORT : 0) | (st.part == R2 ? DOWN : 0) | (w.n % SEGS) << 8;
  const size_t off = (size_t)w.first * SEG + c * 16;
  f.lo = s.w0 + (size_t)g * ge.rb + off;
  f.hi = s.w1 + (size_t)g * ge.rb + off;
  const int rows = (pairs ? 8 : ROWS) * task_stride(ge);    // from one task of the run to the next
  f.step = (ptrdiff_t)rows * ge.rb - (ptrdiff_t)f.nu * UNIT;
  if (FMT == Q4) {
    // groups 2c, 2c + 1 of the unit's eight; words of two groups, from the
    // word that holds the first (a row of an odd number of groups may start
    // in the middle of one)
    const int KG = ge.rb / 32, g0 = w.first * 2 + 2 * c;
    f.groups = KG - g0;
    f.sc_lo = (((s.r0 + g) * (size_t)KG + g0) & ~(size_t)1) * 2;
    f.sc_hi = (((s.r1 + g) * (size_t)KG + g0) & ~(size_t)1) * 2;
    f.sc_step = rows * KG * 2 - f.nu * 16;
    if ((KG & 1) && (g & 1)) f.flags |= ODD;
  }
}

// The stream at the first part from `part` on in which this warp has a task.
// (By value: a reference would keep the caller's copy in memory.)
template <int FMT>
__device__ __noinline__ Feed feed_part(const FewParams &p, Shared *sh, Feed f, int part) {
  const int warp = threadIdx.x >> 5;
  FeedState &st = sh->feed[warp];
  __syncwarp();
  FeedState n = st;
  for (; part < n.limit; ++part) {
    n.g = part < R1 ? part_geo<BF16>(p, part, sh->nact) : part_geo<FMT>(p, part, sh->nact);
    n.j = first_task(n.g, warp);
    if (n.j < n.g.n) break;
  }
  n.part = part;
  f.left = 0;
  if (part < n.limit) feed_run<FMT>(p, sh, n, f);
  __syncwarp();
  st = n;                                   // (every lane the same)
  __syncwarp();
  return f;
}

// The run after the one that is used up
template <int FMT>
__device__ __noinline__ Feed feed_next(const FewParams &p, Shared *sh, Feed f) {
  FeedState &st = sh->feed[threadIdx.x >> 5];
  __syncwarp();
  FeedState n = st;
  n.j += n.run * task_stride(n.g);
  if (n.j >= n.g.n) return feed_part<FMT>(p, sh, f, n.part + 1);
  feed_run<FMT>(p, sh, n, f);
  __syncwarp();
  st = n;
  __syncwarp();
  return f;
}

__device__ __forceinline__ void flush_words(Words &w) {
  if (w.at) {
    st_shared4(w.at, w.w[0]);
    st_shared4(w.at + 16, w.w[1]);
    w.at = 0;
  }
}

// Fetches the next unit (if there is one yet) and closes its group.
template <int FMT, int DEPTH>
__device__ __forceinline__ void feed_step(const FewParams &p, Shared *sh, Feed &f, Words &words, uint32_t ring) {
  if (f.left > 0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t slot = ring + (f.issued % DEPTH) * unit_bytes(FMT);
    // 4-bit pieces: lane (g, c) keeps its 16 bytes so that the eight bytes that
    // the lanes of four rows read at once lie in different banks
    const uint32_t dst = slot + (FMT == Q4 ? g * 64 + ((c ^ (g & 2)) << 4) : lane * 16);
    const int rest = f.left == 1 ? f.flags >> 8 : 0;
    if ((f.flags & FULL) && rest == 0) {
#pragma unroll
      for (int s = 0; s < SEGS; ++s) {
        cp_async16(dst + s * 1024, f.lo + s * SEG);
        cp_async16(dst + s * 1024 + 512, f.hi + s * SEG);
      }
    } else {
      const int n = (rest ? rest : SEGS) - (f.left == 1 && (f.flags & SHORT) ? 1 : 0);
#pragma unroll 1
      for (int s = 0; s < n; ++s) {
        if (f.flags & HAS_LO) cp_async16(dst + s * 1024, f.lo + s * SEG);
        if (f.flags & HAS_HI) cp_async16(dst + s * 1024 + 512, f.hi + s * SEG);
      }
    }
    f.lo += UNIT;
    f.hi += UNIT;
    if (FMT == Q4) {                        // (no shared expert here: every part is of 4-bit rows)
      flush_words(words);
      words.at = slot + ROWS * UNIT + lane * 32;
      if (f.groups > 0) {
        const bool down = f.flags & DOWN;
        const char *const base[4] = {
            static_cast<const char *>(down ? p.s3 : p.s1) + f.sc_lo, static_cast<const char *>(down ? p.b3 : p.b1) + f.sc_lo,
            static_cast<const char *>(down ? p.s3 : p.s2) + f.sc_hi, static_cast<const char *>(down ? p.b3 : p.b2) + f.sc_hi};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          words.w[0][q] = ld_stream(base[q]);
          if ((f.flags & ODD) && f.groups > 1) words.w[1][q] = ld_stream(base[q] + 4);
        }
      }
      f.sc_lo += 16;
      f.sc_hi += 16;
      f.groups -= 8;
    }
    ++f.issued;
    if (--f.left == 0) {
      if (--f.run > 0) {
        f.lo += f.step;
        f.hi += f.step;
        f.left = f.nu;
        if (FMT == Q4) {
          f.sc_lo += f.sc_step;
          f.sc_hi += f.sc_step;
          f.groups += f.nu * 8;
        }
      } else {
        f = feed_next<FMT>(p, sh, f);
      }
    }
  } else if (FMT == Q4) {
    flush_words(words);
  }
  cp_async_commit();
}

// Lets the stream go on into parts before `limit`, and fills it up.
template <int FMT, int DEPTH>
__device__ __noinline__ Feed feed_open(const FewParams &p, Shared *sh, Feed f, uint32_t ring, int limit) {
  FeedState &st = sh->feed[threadIdx.x >> 5];
  __syncwarp();
  const int from = st.part;
  const bool stopped = from >= st.limit;
  __syncwarp();
  st.limit = limit;
  __syncwarp();
  if (stopped) f = feed_part<FMT>(p, sh, f, from);
  Words words{};
#pragma unroll 1
  for (uint32_t i = f.issued - f.used; i < DEPTH; ++i) feed_step<FMT, DEPTH>(p, sh, f, words, ring);
  if (FMT == Q4) flush_words(words);
  return f;
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// with a zero accumulator
__device__ __forceinline__ void mma_s8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
}
// 16 bytes of a token's row, kept in L1.  The rows that this kernel writes
// (codes of x, h) are read after a grid barrier, whose acquire keeps older
// copies out of L1.
__device__ __forceinline__ uint4 ld_l1(const char *p) {
  uint4 v;
  asm volatile("ld.global.ca.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// the larger magnitude, NaN above all
__device__ __forceinline__ float abs_max(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu));
}
__device__ __forceinline__ float silu_f(float g) { return g / (1.f + expf(-g)); }

constexpr float DIGITS_MAX = 32512.f;       // 127 * 256: the high digit stays in [-127, 127]

// bytes of the token row (4-bit: of one digit of it) per byte of the weight row
template <int FMT>
__host__ __device__ constexpr int ratio_of() {
  return FMT == Q4 ? 2 : 1;
}
// B operand of one segment: 16 bytes of the token row (bf16 phase 2: and of its
// low part).  4-bit: a segment is two groups of 64 codes; 16 bytes of each
// digit per group.
template <int FMT, bool LO>
struct BSeg {
  uint4 v[FMT == Q4 ? 2 : 1][LO || FMT == Q4 ? 2 : 1];
};

// row: this lane's place in the segment's stretch of the token row; second:
// bytes from there to the low part or digit; left: bytes of the weight row
// from the segment on.  CHECK: the segment may reach past the row's end.
template <int FMT, bool LO, bool CHECK>
__device__ __forceinline__ void load_b(BSeg<FMT, LO> &bv, const char *row, size_t second, int left, int c) {
#pragma unroll
  for (int q = 0; q < (FMT == Q4 ? 2 : 1); ++q) {
    const bool ok = !CHECK || (FMT == Q4 ? q * 32 : c * 16) < left;
#pragma unroll
    for (int l = 0; l < (LO || FMT == Q4 ? 2 : 1); ++l)
      bv.v[q][l] = ok ? ld_l1(row + q * 64 + (l ? second : 0)) : make_uint4(0u, 0u, 0u, 0u);
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

// One segment of the 16 rows times the tokens.  a: this lane's place in the
// segment's slots (4-bit: row g's); left: bytes of the rows from the segment
// on.  4-bit: sw, the lane's scale words of the segment (s and b of row g, of
// row g + 8, two groups each), and gs(n, q, j), the sum of token 2c + j of
// block n over the segment's group q.
template <int FMT, bool LO, int NB, bool CHECK, class Sums>
__device__ __forceinline__ void consume(Acc<FMT, NB> &acc, const BSeg<FMT, LO> (&bv)[NB], int left, const uint8_t *a,
                                        int g, int c, const uint32_t (&sw)[4], Sums gs) {
  if constexpr (FMT != Q4) {
    uint4 lo = *reinterpret_cast<const uint4 *>(a), hi = *reinterpret_cast<const uint4 *>(a + 512);
    if (CHECK && c * 16 >= left) lo = hi = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
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
      const int half = (q ^ ((g >> 1) & 1)) * 32 + c * 8;
      const uint2 lo = *reinterpret_cast<const uint2 *>(a + half);
      const uint2 hi = *reinterpret_cast<const uint2 *>(a + 512 + half);
      // a word's codes 0, 2, 4, 6 and 1, 3, 5, 7: the digits lie in that order
      constexpr uint32_t nib = 0x0F0F0F0Fu;
      const uint32_t l0 = lo.x & nib, l1 = (lo.x >> 4) & nib, l2 = lo.y & nib, l3 = (lo.y >> 4) & nib;
      const uint32_t h0 = hi.x & nib, h1 = (hi.x >> 4) & nib, h2 = hi.y & nib, h3 = (hi.y >> 4) & nib;
      const float s_lo = __uint_as_float(q ? sw[0] & 0xFFFF0000u : sw[0] << 16);
      const float s_hi = __uint_as_float(q ? sw[2] & 0xFFFF0000u : sw[2] << 16);
      const float b_lo = __uint_as_float(q ? sw[1] & 0xFFFF0000u : sw[1] << 16);
      const float b_hi = __uint_as_float(q ? sw[3] & 0xFFFF0000u : sw[3] << 16);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        int d[2][4];
#pragma unroll
        for (int l = 0; l < 2; ++l) {
          const uint4 b = bv[n].v[q][l];
          mma_s8_first(d[l], l0, h0, l1, h1, b.x, b.y);
          mma_s8(d[l], l2, h2, l3, h3, b.z, b.w);
        }
        const float g0 = gs(n, q, 0), g1 = gs(n, q, 1);
        float(&t)[4] = acc.f[n][q];
        t[0] = fmaf(s_lo, (float)(d[0][0] * 256 + d[1][0]), fmaf(b_lo, g0, t[0]));
        t[1] = fmaf(s_lo, (float)(d[0][1] * 256 + d[1][1]), fmaf(b_lo, g1, t[1]));
        t[2] = fmaf(s_hi, (float)(d[0][2] * 256 + d[1][2]), fmaf(b_hi, g0, t[2]));
        t[3] = fmaf(s_hi, (float)(d[0][3] * 256 + d[1][3]), fmaf(b_hi, g1, t[3]));
      }
    }
  }
}

// n-th set bit of a mask (the mask has more than n)
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
  for (int i = 0; i < n; ++i) m &= m - 1;
  return __ffs(m) - 1;
}

struct Cursor {
  int e, rows, row0, b, kp;                 // row0: first row of h / y; b: row block; kp: part of K
  uint32_t mask;
};

__device__ __forceinline__ Cursor cursor_of(const FewParams &p, const Shared *sh, const Geo &g, int part, int task) {
  Cursor cu;
  const Task t = task_of(g, task);
  cu.kp = t.kp;
  cu.b = t.b;
  if (part < R1) {
    cu.e = 0;
    cu.mask = (1u << p.T) - 1u;
    cu.row0 = 0;
    cu.rows = p.T;
  } else {
    cu.e = sh->act[t.i];
    cu.mask = sh->mask[cu.e];
    cu.row0 = sh->row0[t.i];
    cu.rows = sh->row0[t.i + 1] - cu.row0;
  }
  return cu;
}

// Row r of a task's token operand.  A row past the task's last repeats the
// last: each token is a column of its own, and those columns are not stored.
template <int FMT, bool PHASE2>
__device__ __forceinline__ const char *b_row(const FewParams &p, const Cursor &cu, int part, int r) {
  r = min(r, cu.rows - 1);
  if (!PHASE2) {
    const int t = part == S1 ? r : nth_bit(cu.mask, r);
    return FMT == BF16 ? reinterpret_cast<const char *>(p.x + (size_t)t * p.d)
                       : reinterpret_cast<const char *>(p.xq + (size_t)t * (FMT == Q4 ? 2 : 1) * p.d);
  }
  if (part == S2) return reinterpret_cast<const char *>(p.hs + (size_t)r * p.Fs);
  return FMT == BF16 ? reinterpret_cast<const char *>(p.h + (size_t)(cu.row0 + r) * p.F)
                     : reinterpret_cast<const char *>(p.hq + (size_t)(cu.row0 + r) * (FMT == Q4 ? 2 : 1) * p.F);
}

// 4-bit: its sums over the groups
template <bool PHASE2>
__device__ __forceinline__ const float *g_row(const FewParams &p, const Cursor &cu, int r) {
  r = min(r, cu.rows - 1);
  return PHASE2 ? p.hg + (size_t)(cu.row0 + r) * (p.F / 64) : p.xg + (size_t)nth_bit(cu.mask, r) * (p.d / 64);
}

// What a finished value is multiplied by: the row's scale (of the token in
// phase 1, of the row of h in phase 2) and with 8-bit weights the channel's.
// Fetched when a task begins, for the value that the thread will hold at its end.
struct Scale {
  float v, u;
};
template <int FMT, bool PHASE2>
__device__ __forceinline__ float row_scale(const FewParams &p, const Cursor &cu, int tok) {
  if (FMT == BF16 || tok >= cu.rows) return 1.f;
  if (!PHASE2) return __ldcg(p.xs + nth_bit(cu.mask, tok));
  const uint32_t top = __ldcg(p.rowmax + cu.row0 + tok);
  return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u)
                            : __fdiv_rn(__uint_as_float(top), FMT == Q4 ? DIGITS_MAX : 127.f);
}
template <int FMT, bool PHASE2>
__device__ __forceinline__ Scale scale_of(const FewParams &p, const Cursor &cu, bool pairs, int col, float row) {
  Scale s{row, row};
  if (FMT == I8 && col < (PHASE2 ? p.d : p.F)) {
    const size_t r0 = (size_t)cu.e * (PHASE2 ? p.d : p.w_stride) + col;
    s.v *= __ldg(static_cast<const float *>(PHASE2 ? p.s3 : p.s1) + r0);
    if (pairs) s.u *= __ldg(static_cast<const float *>(p.s2) + r0);
  }
  return s;
}

// What becomes of one finished value: column col of token tok (with its up
// projection u where the task holds pairs).  Returns the magnitude of the
// stored h (8-bit and 4-bit weights: the row maxima are taken from it).
template <int FMT, bool PHASE2>
__device__ __forceinline__ float emit(const FewParams &p, const Cursor &cu, int part, bool pairs, int col, int tok, float v,
                                      float u, Scale s) {
  const int N = PHASE2 ? p.d : (part == S1 ? p.Fs : p.F);
  if (tok >= cu.rows || col >= N) return 0.f;
  const size_t row = (size_t)cu.row0 + tok;
  if (FMT != BF16) {
    v *= s.v;
    if (pairs) u *= s.u;
  }
  if (PHASE2) {
    p.y[(part == S2 ? (size_t)p.ksplit * p.y_rows + tok : (size_t)cu.kp * p.y_rows + row) * p.d + col] = v;
    return 0.f;
  }
  if (pairs) v = silu_f(v) * u;
  else v = v < 0.f ? 0.f : v;               // a NaN stays one
  if (FMT == Q4) {
    p.hf[row * p.F + col] = v;
    return v;
  }
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  uint16_t *h = part == S1 ? p.hs + (size_t)tok * p.Fs + col : p.h + row * p.F + col;
  *h = *reinterpret_cast<const uint16_t *>(&hi);
  if (FMT == BF16) {
    const float rest = v - __bfloat162float(hi);
    const __nv_bfloat16 lo = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
    h[part == S1 ? p.hs_lo : p.h_lo] = *reinterpret_cast<const uint16_t *>(&lo);
  }
  return __bfloat162float(hi);
}

// One barrier of a group's warps (of the two groups, in turn numbers 1 and 2)
__device__ __forceinline__ void group_sync() {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + (threadIdx.x >> 5) / GW), "n"(32 * GW) : "memory");
}

// A run of a warp's tasks: `run` of them, every by-th row block from cu.b on, of
// one expert (and part of K): the same tokens, the same place in K.  NB blocks
// of eight tokens, MAXNB the most of any run (the layout of the meeting place).
// RFMT: the routed experts' format, which the stream may go on to.
template <int FMT, int RFMT, bool PHASE2, int NB, int MAXNB, int DEPTH>
__device__ __noinline__ Feed consume_run(const FewParams &p, Shared *sh, uint8_t *ring_ptr, Feed f, uint32_t &red_it_ref,
                                         int part, const Geo &geo, Cursor cu, int run) {
  uint32_t red_it = red_it_ref;
  Words words{};
  constexpr bool LO = PHASE2 && FMT == BF16;
  constexpr int R = ratio_of<FMT>();
  const bool solo = geo.solo;
  const int rb = geo.rb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(ring_ptr);
  const size_t lo_bytes = FMT == Q4 ? (PHASE2 ? p.F : p.d) : 2 * (part == S2 ? p.hs_lo : p.h_lo);   // to the low part or digit
  const bool odd_groups = FMT == Q4 && (rb / 32 & 1) && (lg & 1);
  const bool pairs = !PHASE2 && (part == S1 || p.swiglu);
  const bool top_of_h = FMT != BF16 && part == R1;
  const int by = task_stride(geo);
  const int cols = pairs ? 8 : ROWS;        // outputs of a task
  const int KG = rb / 32;                   // 4-bit: groups of a row
  // long rows: this thread of its group sums up output (value) number id and,
  // with more than eight tokens, maybe one 256 further
  const int id0 = threadIdx.x % (32 * GW);
  constexpr bool second = NB > 1;
  const Span w = warp_span(geo, cu.kp, warp);
  const char *rowp[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) rowp[n] = b_row<FMT, PHASE2>(p, cu, part, lg + 8 * n) + c * 16 + (size_t)w.first * SEG * R;
  const float *sums[NB];
  if constexpr (FMT == Q4) {
#pragma unroll
    for (int n = 0; n < NB; ++n) sums[n] = g_row<PHASE2>(p, cu, lg + 8 * n) + 2 * w.first + c;
  }
  // whole units of the warp's span: the rest, and a last segment that is not
  // whole, go through the checked path
  const bool uneven = rb % SEG != 0 && w.first + w.n == geo.ns;
  const int whole = (w.n - (uneven ? 1 : 0)) / SEGS;
  float row_sc[NB][2];                      // solo: of tokens 2c, 2c + 1 of each block
  if (FMT != BF16 && solo) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      row_sc[n][0] = row_scale<FMT, PHASE2>(p, cu, 8 * n + 2 * c);
      row_sc[n][1] = row_scale<FMT, PHASE2>(p, cu, 8 * n + 2 * c + 1);
    }
  }
  for (int r = 0; r < run; ++r, cu.b += by) {
    Acc<FMT, NB> acc;
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc.f[n][0][i] = acc.f[n][1][i] = 0;
    // the scales of what this thread will hold at the end
    Scale sc[2]{{1.f, 1.f}, {1.f, 1.f}};
    const int id = (id0 + 64 * red_it) % (32 * GW);     // (other warps from task to task)
    if (FMT == I8) {
      if (solo) {
        sc[0] = scale_of<FMT, PHASE2>(p, cu, pairs, cu.b * cols + lg, 1.f);
        if (!pairs) sc[1] = scale_of<FMT, PHASE2>(p, cu, pairs, cu.b * cols + lg + 8, 1.f);
      } else if (id < cols * 8) {
        sc[0] = scale_of<FMT, PHASE2>(p, cu, pairs, cu.b * cols + (id & (cols - 1)),
                                      row_scale<FMT, PHASE2>(p, cu, id >> (pairs ? 3 : 4)));
      }
    }
    const char *bp[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) bp[n] = rowp[n];
    for (int u = 0; u * SEGS < w.n; ++u) {
      const uint8_t *slot = ring_ptr + (f.used % DEPTH) * unit_bytes(RFMT);
      const uint8_t *a = FMT == Q4 ? slot + lg * 64 : slot + lane * 16;
      float gsum[NB][2] = {};             // 4-bit: sums of the lane's token rows over groups c, c + 4 of the unit
      if constexpr (FMT == Q4) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int at = 2 * (w.first + u * SEGS) + c;
          gsum[n][0] = at < KG ? ld_l1_f32(sums[n] + u * 8) : 0.f;
          gsum[n][1] = at + 4 < KG ? ld_l1_f32(sums[n] + u * 8 + 4) : 0.f;
        }
      }
      auto segment = [&](int s, const BSeg<FMT, LO>(&bv)[NB], int left, auto check) {
        uint32_t sw[4] = {0u, 0u, 0u, 0u};
        if constexpr (FMT == Q4) {
          const uint4 *t = reinterpret_cast<const uint4 *>(slot + ROWS * UNIT + (lg * 4 + s) * 32);
          const uint4 x = t[0];
          sw[0] = x.x; sw[1] = x.y; sw[2] = x.z; sw[3] = x.w;
          if (odd_groups) {
            const uint4 y = t[1];
            sw[0] = __funnelshift_r(x.x, y.x, 16); sw[1] = __funnelshift_r(x.y, y.y, 16);
            sw[2] = __funnelshift_r(x.z, y.z, 16); sw[3] = __funnelshift_r(x.w, y.w, 16);
          }
        }
        consume<FMT, LO, NB, decltype(check)::value>(
            acc, bv, left, a + s * 1024, lg, c, sw, [&](int n, int q, int i) {
              // group 2 s + q of the unit, held by the lanes of one quad column
              return __shfl_sync(0xffffffffu, s < 2 ? gsum[n][0] : gsum[n][1], c * 8 + i * 4 + (2 * s + q) % 4);
            });
      };
      if (u < whole) {
        if constexpr (FMT == Q4) {
          // (rolled: the body is long, and fetching instructions would cost more);
          // the token operand is a segment ahead
          BSeg<FMT, LO> bv[NB], next[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n) load_b<FMT, LO, false>(bv[n], bp[n], lo_bytes, SEG, c);
          cp_async_wait<DEPTH - 1>();
          __syncwarp();
#pragma unroll 1
          for (int s = 0; s < SEGS; ++s) {
            const int ahead = min(s + 1, SEGS - 1);
#pragma unroll
            for (int n = 0; n < NB; ++n)
              load_b<FMT, LO, false>(next[n], bp[n] + ahead * SEG * R, lo_bytes, SEG, c);
            segment(s, bv, SEG, std::false_type{});
#pragma unroll
            for (int n = 0; n < NB; ++n) bv[n] = next[n];
          }
        } else {
          // the token operand is on its way while the weights are waited for
          constexpr int HELD = LO && NB > 1 ? 2 : SEGS;
          BSeg<FMT, LO> bv[HELD][NB];
#pragma unroll
          for (int s0 = 0; s0 < SEGS; s0 += HELD) {
#pragma unroll
            for (int s = 0; s < HELD; ++s)
#pragma unroll
              for (int n = 0; n < NB; ++n)
                load_b<FMT, LO, false>(bv[s][n], bp[n] + (s0 + s) * SEG * R, lo_bytes, SEG, c);
            if (s0 == 0) cp_async_wait<DEPTH - 1>();
#pragma unroll
            for (int s = 0; s < HELD; ++s) segment(s0 + s, bv[s], SEG, std::false_type{});
          }
        }
      } else {
        const int n_seg = min(SEGS, w.n - u * SEGS);
        const int left = rb - (w.first + u * SEGS) * SEG;        // bytes of the row from here on
        cp_async_wait<DEPTH - 1>();
        if (FMT == Q4) __syncwarp();
#pragma unroll 1
        for (int s = 0; s < n_seg; ++s) {
          BSeg<FMT, LO> bv[NB];
#pragma unroll
          for (int n = 0; n < NB; ++n)
            load_b<FMT, LO, true>(bv[n], bp[n] + s * SEG * R, lo_bytes, left - s * SEG, c);
          segment(s, bv, left - s * SEG, std::true_type{});
        }
      }
      if (FMT == Q4) __syncwarp();
#pragma unroll
      for (int n = 0; n < NB; ++n) bp[n] += UNIT * R;
      ++f.used;
      feed_step<RFMT, DEPTH>(p, sh, f, words, ring);
    }
    if (solo) {
      // accumulators 0, 1: row g, tokens 2c, 2c + 1; 2, 3: row g + 8
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = 8 * n + 2 * c + i;
          const float v0 = (float)(acc.f[n][0][i] + acc.f[n][1][i]);
          const float v1 = (float)(acc.f[n][0][i + 2] + acc.f[n][1][i + 2]);
          const float rs = FMT != BF16 ? row_sc[n][i] : 1.f;
          float m = emit<FMT, PHASE2>(p, cu, part, pairs, cu.b * cols + lg, tok, v0, v1, {sc[0].v * rs, sc[0].u * rs});
          if (!pairs)
            m = abs_max(m, emit<FMT, PHASE2>(p, cu, part, pairs, cu.b * cols + lg + 8, tok, v1, 0.f,
                                             {sc[1].v * rs, 1.f}));
          if (top_of_h) {
            uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lg == 0 && tok < cu.rows) atomicMax(p.rowmax + cu.row0 + tok, top);
          }
        }
      }
    } else {
      // the group's partial results meet; two buffers in turn, so one
      // barrier per task keeps writers and readers apart
        uint32_t(*red)[MAXNB][32][4] = &reinterpret_cast<Partial<MAXNB> *>(partials(sh))->red[red_it & 1u][warp / GW * GW];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const auto sum = acc.f[n][0][i] + acc.f[n][1][i];
          if constexpr (FMT == I8) v[i] = (uint32_t)sum;
          else v[i] = __float_as_uint(sum);
        }
        *reinterpret_cast<uint4 *>(red[warp % GW][n][lane]) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      group_sync();
      ++red_it;
      // value (row, token) of the task: accumulator i of lane 4 (row % 8) + (token % 8) / 2
      auto total = [&](int row, int tok) {
        const int ln = (row & 7) * 4 + ((tok & 7) >> 1), i = (tok & 1) + (row >> 3) * 2, n = tok >> 3;
        if (FMT == I8) {
          int v = 0;
#pragma unroll
          for (int q = 0; q < GW; ++q) v += (int)red[q][n][ln][i];
          return (float)v;
        }
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < GW; ++q) v += __uint_as_float(red[q][n][ln][i]);
        return v;
      };
      const int most = cols * 8 * (second ? 2 : 1);               // (at most the group's threads)
      if (id < most) {
        const int tok = id >> (pairs ? 3 : 4), q = id & (cols - 1);
        if (FMT != BF16 && (FMT == Q4 || id >= cols * 8))
          sc[0] = scale_of<FMT, PHASE2>(p, cu, pairs, cu.b * cols + q, row_scale<FMT, PHASE2>(p, cu, tok));
        float m = 0.f;
        if (tok < cu.rows)
          m = emit<FMT, PHASE2>(p, cu, part, pairs, cu.b * cols + q, tok, total(q, tok), pairs ? total(q + 8, tok) : 0.f,
                                sc[0]);
        if (top_of_h) {
          // the row's largest |h|: over the task's columns (8 or 16 neighbouring lanes), then the grid
          uint32_t top = __float_as_uint(m) & 0x7FFFFFFFu;
          for (int o = 1; o < cols; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (q == 0 && tok < cu.rows) atomicMax(p.rowmax + cu.row0 + tok, top);
        }
      }
    }
  }
  if (RFMT == Q4) flush_words(words);
  red_it_ref = red_it;
  return f;
}

// The block's tasks of one part (of phase 1 or 2), run by run
template <int FMT, int RFMT, bool PHASE2, int NB, int DEPTH>
__device__ __noinline__ Feed consume_part(const FewParams &p, Shared *sh, uint8_t *ring_ptr, Feed f, uint32_t &red_it,
                                          int part) {
  const Geo g = part_geo<FMT>(p, part, sh->nact);
  const int warp = threadIdx.x >> 5;
  for (int j = first_task(g, warp); j < g.n;) {
    const Cursor cu = cursor_of(p, sh, g, part, g.first + j);
    const int run = run_of(g, j, cu.b);
    if (NB > 1 && cu.rows > 8) f = consume_run<FMT, RFMT, PHASE2, NB, NB, DEPTH>(p, sh, ring_ptr, f, red_it, part, g, cu, run);
    else f = consume_run<FMT, RFMT, PHASE2, 1, NB, DEPTH>(p, sh, ring_ptr, f, red_it, part, g, cu, run);
    j += run * task_stride(g);
  }
  return f;
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
  double(*sums)[MAX_T] = reinterpret_cast<double(*)[MAX_T]>(partials(sh));
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
    __syncthreads();
    for (int i = threadIdx.x; i < at_once * p.T; i += CT) {
      const int t = i / at_once, q = i - t * at_once;
      double s = 0.0;
      for (int j = 0; j < per; ++j) s += sums[q * per + j][t];
      if (e0 + q < p.E) p.logits[(size_t)t * p.E + e0 + q] = s;
    }
    __syncthreads();
  }
}

constexpr int EPL = kMaxExperts / 32;

// One token's choice from its row of `prob` (softmax: shifted logits, made
// probabilities here; sigmoid: probabilities); ids and weights to shared
// memory.  A warp; expert lane + 32 j.
__device__ __forceinline__ void choose(const FewParams &p, Shared *sh, int t, double *prob, int lane) {
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
        key[j] = key_of(prob[e] + (double)sh->bias[e]);
      }
    }
    // group score = sum of the two largest selection scores in the group
    const int G = E / p.n_group;
    unsigned long long gkey = 0;
    if (lane < p.n_group) {
      unsigned long long b1 = 0, b2 = 0;
#pragma unroll 4
      for (int q = 0; q < G; ++q) {
        const unsigned long long v = key_of(prob[lane * G + q] + (double)sh->bias[lane * G + q]);
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
    const int inv = (65536 + G - 1) / G;               // e / G = e inv >> 16 for every e < E <= 256
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (e < E && !((keep >> (e * inv >> 16)) & 1u)) key[j] = min(key[j], LOWEST);
    }
  }
  // the lane's experts in order (Batcher's network of 19 exchanges, mostly
  // side by side), so that a round looks at each lane's first only
  int at[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) at[j] = lane + 32 * j;
  if (E > 32) {
    constexpr int net[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
    static_assert(EPL == 8, "the network sorts eight");
#pragma unroll
    for (int q = 0; q < 19; ++q) {
      const int a = net[q][0], b = net[q][1];
      const bool swap = key[b] > key[a] || (key[b] == key[a] && at[b] < at[a]);
      const unsigned long long ka = key[a];
      const int ia = at[a];
      key[a] = swap ? key[b] : ka;
      at[a] = swap ? at[b] : ia;
      key[b] = swap ? ka : key[b];
      at[b] = swap ? ia : at[b];
    }
  }

  int my_e = 0x7fffffff;
#pragma unroll 1
  for (int r = 0; r < p.k; ++r) {
    const int bi = warp_argmax(key[0], key[0] ? at[0] : 0x7fffffff);
    if (bi == at[0]) {                                 // taken: the lane's next moves up
#pragma unroll
      for (int j = 0; j + 1 < EPL; ++j) {
        key[j] = key[j + 1];
        at[j] = at[j + 1];
      }
      key[EPL - 1] = 0ull;
    }
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
__device__ __noinline__ void make_plan(const FewParams &p, Shared *sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  static_assert(sizeof(Partial<1>) >= 8 * kMaxExperts * sizeof(double) &&
                    sizeof(Partial<2>) >= MAX_T * kMaxExperts * sizeof(double),
                "a row of probabilities per token");
  double *prob = reinterpret_cast<double *>(partials(sh));
  if (tid < kMaxExperts) sh->mask[tid] = 0u;
  static_assert(CT >= kMaxExperts && CW >= MAX_T, "a thread per expert, a warp per token");
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
      if (p.bias) l += (double)sh->bias[i % p.E];
    } else {
      l = 1.0 / (1.0 + exp(-l));
    }
    prob[i] = l;
  }
  __syncthreads();
  if (const int t = warp; t < p.T) choose(p, sh, t, prob + (size_t)t * p.E, lane);
  __syncthreads();
  const int slots = p.T * p.k;
#pragma unroll 1
  for (int i = tid; i < slots; i += CT) {
    const int e = sh->sel_id[i];
    if (e >= 0) atomicOr(&sh->mask[e], 1u << (i / p.k));
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid < p.E) {
    double s = 0.0;
    for (int t = 0; t < p.T; ++t) s += prob[(size_t)t * p.E + tid];
    p.prob_sum[tid] = (float)s;
  }
  // thread e: expert e.  In-order dropping: the first `cap` tokens stay
  uint32_t m = tid < kMaxExperts ? sh->mask[tid] : 0u;
  if (tid < kMaxExperts) sh->raw[tid] = (uint8_t)__popc(m);
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
  if (tid < kMaxExperts) sh->mask[tid] = m;
  __syncthreads();
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
  __syncthreads();
}

// What the call returns beside the output; one block, while it waits
__device__ __forceinline__ void write_choice(const FewParams &p, const Shared *sh) {
  const int e = threadIdx.x;
  for (int i = e; i < p.T * p.k; i += CT) {
    p.ids[i] = sh->sel_id[i];
    p.wts[i] = sh->sel_w[i];
  }
  if (e < p.E) {
    const int raw = sh->raw[e], kept = __popc(sh->mask[e]);
    p.raw_counts[e] = raw;
    p.kept_counts[e] = kept;
    if (raw > kept) atomicAdd(p.dropped, raw - kept);
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

// 16-bit integers of 8 elements of a row with largest magnitude `top`, as two
// digits, in the order in which a word's codes unpack (0, 2, 4, 6, 1, 3, 5, 7);
// returns their sum.
__device__ __forceinline__ int digits8(const float (&x)[8], uint32_t top, uint2 &hi, uint2 &lo) {
  hi = lo = make_uint2(0u, 0u);
  if (top == 0u || top >= 0x7F800000u) return 0;
  float a = __uint_as_float(top);
  const float pre = a < 0x1p-60f ? 0x1p64f : (a > 0x1p100f ? 0x1p-32f : 1.f);
  a *= pre;
  const float r = __fdiv_rn(DIGITS_MAX, a);
  int v[8], sum = 0;
  uint32_t t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __float_as_int(fmaf(x[i] * pre, r, 12582912.f)) - 0x4B400000;   // rounded to the nearest, |v| <= 32512
    t[i] = (uint32_t)(v[i] + 128);          // its second byte: (v + 128) >> 8
    sum += v[i];
  }
  auto low = [](uint32_t a0, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a0, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  };
  auto next = [](uint32_t a0, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a0, b, 0x0051), __byte_perm(c, d, 0x0051), 0x5410);
  };
  lo = make_uint2(low(v[0], v[2], v[4], v[6]), low(v[1], v[3], v[5], v[7]));
  hi = make_uint2(next(t[0], t[2], t[4], t[6]), next(t[1], t[3], t[5], t[7]));
  return sum;
}

// One step of a digit pass: eight elements per thread (live ones: whole groups
// of eight neighbouring threads), vector i of a row of K.  Called by whole warps.
__device__ __forceinline__ void store_digits(const float (&x)[8], uint32_t top, bool live, int i, int K, int8_t *digits,
                                             float *sums) {
  uint2 hi, lo;
  int sum = digits8(x, top, hi, lo);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (live) {
    reinterpret_cast<uint2 *>(digits)[i] = hi;
    reinterpret_cast<uint2 *>(digits + K)[i] = lo;
    if ((i & 7) == 0) sums[i >> 3] = (float)sum;
  }
}

// token rows: one block each, from the last block down (the router's units
// start at the first)
template <int FMT>
__device__ __forceinline__ void quantize_x(const FewParams &p, Shared *sh) {
  uint32_t *scratch = partials(sh);
  for (int t = (int)gridDim.x - 1 - (int)blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4 *row = reinterpret_cast<const uint4 *>(p.x + (size_t)t * p.d);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < p.d / 8; i += CT) {
      const uint4 v = __ldg(row + i);
      m = abs_max2(v.x, abs_max2(v.y, abs_max2(v.z, abs_max2(v.w, m))));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < CW; ++w) m = max(m, scratch[w]);
    if (FMT == I8) {
      for (int i = threadIdx.x; i < p.d / 8; i += CT)
        reinterpret_cast<uint2 *>(p.xq + (size_t)t * p.d)[i] = codes8(__ldg(row + i), m);
    } else {
      for (int i0 = 0; i0 < p.d / 8; i0 += CT) {
        const int i = i0 + threadIdx.x;
        const bool live = i < p.d / 8;
        const uint4 v = live ? __ldg(row + i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float x[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
        store_digits(x, m, live, i, p.d, p.xq + (size_t)t * 2 * p.d, p.xg + (size_t)t * (p.d / 64));
      }
    }
    if (threadIdx.x == 0)
      p.xs[t] = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(m), FMT == Q4 ? DIGITS_MAX : 127.f);
    __syncthreads();                        // the scratch has been read
  }
}

// rows of h, all blocks together
template <int FMT>
__device__ __forceinline__ void quantize_h(const FewParams &p, const Shared *sh) {
  const int rows = sh->row0[sh->nact], nv = p.F / 8;
  const long long n = (long long)rows * nv, step = (long long)gridDim.x * CT;
  for (long long i0 = (long long)blockIdx.x * CT; i0 < n; i0 += step) {
    const long long i = i0 + threadIdx.x;
    const bool live = i < n;
    const int r = live ? (int)(i / nv) : 0;
    const uint32_t top = live ? __ldcg(p.rowmax + r) : 0u;
    if (FMT == I8) {
      if (live) reinterpret_cast<uint2 *>(p.hq)[i] = codes8(__ldcg(reinterpret_cast<const uint4 *>(p.h) + i), top);
    } else {
      const float4 *src = reinterpret_cast<const float4 *>(p.hf) + 2 * i;
      const float4 u = live ? __ldcg(src) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 v = live ? __ldcg(src + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      store_digits(x, top, live, (int)(i - (long long)r * nv), p.F, p.hq + (size_t)r * 2 * p.F, p.hg + (size_t)r * (p.F / 64));
    }
  }
}

// out[t] = sum_j w_j y[slot_row] in slot order (+ the shared expert's row), 4
// columns per thread, the loads of four slots (and their parts of K) in flight
// together
__device__ __forceinline__ void combine(const FewParams &p, const Shared *sh, int ks) {
  const int nv = p.d / 4;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // a warp's 32 vectors are neighbours, the warps' pieces go round the blocks
  const int lane = threadIdx.x & 31;
  for (int i = (blockIdx.x + gridDim.x * (threadIdx.x >> 5)) * 32 + lane; i < p.T * nv; i += gridDim.x * CT) {
    const int t = i / nv, c = i - t * nv;
    float4 a = zero, shared = zero;
    if (p.Fs) shared = __ldcg(reinterpret_cast<const float4 *>(p.y + ((size_t)p.ksplit * p.y_rows + t) * p.d) + c);
#pragma unroll 1
    for (int j0 = 0; j0 < p.k; j0 += 4) {
      float4 v[4][MAX_KSPLIT];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = j0 + u < p.k ? sh->slot_row[t * p.k + j0 + u] : -1;
#pragma unroll
        for (int q = 0; q < MAX_KSPLIT; ++q)
          v[u][q] = row >= 0 && q < ks
                        ? __ldcg(reinterpret_cast<const float4 *>(p.y + ((size_t)q * p.y_rows + row) * p.d) + c)
                        : zero;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (j0 + u >= p.k || sh->slot_row[t * p.k + j0 + u] < 0) continue;
        const float w = sh->sel_w[t * p.k + j0 + u];
        float4 s = v[u][0];
#pragma unroll
        for (int q = 1; q < MAX_KSPLIT; ++q)
          s = make_float4(s.x + v[u][q].x, s.y + v[u][q].y, s.z + v[u][q].z, s.w + v[u][q].w);
        a = make_float4(fmaf(w, s.x, a.x), fmaf(w, s.y, a.y), fmaf(w, s.z, a.z), fmaf(w, s.w, a.w));
      }
    }
    a = make_float4(a.x + shared.x, a.y + shared.y, a.z + shared.z, a.w + shared.w);
    *reinterpret_cast<uint2 *>(p.out + (size_t)t * p.d + 4 * c) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

template <int FMT, int TP>
__global__ void __launch_bounds__(CT, 1) few_kernel(const __grid_constant__ FewParams p) {
  constexpr int NB = TP > 8 ? 2 : 1, DEPTH = depth_of(FMT, TP);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *ring_ptr = smem_raw + (threadIdx.x >> 5) * DEPTH * unit_bytes(FMT);      // this warp's
  const uint32_t ring = smem_u32(ring_ptr);
  Shared *sh = reinterpret_cast<Shared *>(smem_raw + CW * DEPTH * unit_bytes(FMT));
  volatile int *abort_flag = &sh->abort_flag;
  if (threadIdx.x == 0) {
    sh->abort_flag = 0;
    sh->nact = 0;
    if (blockIdx.x == 0) *p.dropped = 0;
  }
  if ((threadIdx.x & 31) == 0) {
    FeedState &st = sh->feed[threadIdx.x >> 5];
    st.part = st.limit = p.Fs ? S1 : R1;
  }
  if (threadIdx.x < kMaxExperts) sh->bias[threadIdx.x] = p.bias && threadIdx.x < p.E ? __ldg(p.bias + threadIdx.x) : 0.f;
  __syncthreads();
  Feed feed{};
  uint32_t red_it = 0;
  constexpr bool SHARED = FMT != Q4;        // (4-bit layers have no shared expert)
  if constexpr (SHARED)
    if (p.Fs) feed = feed_open<FMT, DEPTH>(p, sh, feed, ring, R1);
  if (FMT != BF16) {
    quantize_x<FMT>(p, sh);
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < p.T * p.k; i += CT) p.rowmax[i] = 0u;
  }
  route_logits<TP>(p, sh);
  if constexpr (SHARED)
    if (p.Fs) feed = consume_part<BF16, FMT, false, NB, DEPTH>(p, sh, ring_ptr, feed, red_it, S1);
  grid_arrive(p.bar);
  grid_wait(p.bar, abort_flag, p);
  make_plan(p, sh);
  feed = feed_open<FMT, DEPTH>(p, sh, feed, ring, END);
  if constexpr (SHARED)
    if (p.Fs) feed = consume_part<BF16, FMT, true, NB, DEPTH>(p, sh, ring_ptr, feed, red_it, S2);
  feed = consume_part<FMT, FMT, false, NB, DEPTH>(p, sh, ring_ptr, feed, red_it, R1);
  grid_arrive(p.bar + 8);
  grid_wait(p.bar + 8, abort_flag, p);
  if (FMT != BF16) {
    quantize_h<FMT>(p, sh);
    grid_arrive(p.bar + 16);
    grid_wait(p.bar + 16, abort_flag, p);
  }
  feed = consume_part<FMT, FMT, true, NB, DEPTH>(p, sh, ring_ptr, feed, red_it, R2);
  grid_arrive(p.bar + 24);
  if (blockIdx.x == 0) write_choice(p, sh);
  slot_rows(p, sh);
  grid_wait(p.bar + 24, abort_flag, p);
  combine(p, sh, part_geo<FMT>(p, R2, sh->nact).ks);
  cp_async_wait<0>();
}

template <int FMT, int TP>
__host__ constexpr size_t smem_bytes() {
  return (size_t)CW * depth_of(FMT, TP) * unit_bytes(FMT) + sizeof(Shared) +
         (TP > 8 ? sizeof(Partial<2>) : sizeof(Partial<1>));
}

template <int FMT, int TP>
cudaError_t run(const FewParams &p, cudaStream_t s) {
  const size_t smem = smem_bytes<FMT, TP>();
  auto kern = few_kernel<FMT, TP>;
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  note_launch();
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;      // the blocks wait for one another
  attr[0].val.cooperative = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = sm_count();
  cfg.blockDim = CT;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}
static_assert(smem_bytes<BF16, 8>() <= SMEM_LIMIT && smem_bytes<BF16, 16>() <= SMEM_LIMIT &&
                  smem_bytes<Q4, 8>() <= SMEM_LIMIT && smem_bytes<Q4, 16>() <= SMEM_LIMIT,
              "shared memory");

template <int FMT>
cudaError_t run_t(const FewParams &p, cudaStream_t s) {
  if (p.T <= 1) return run<FMT, 1>(p, s);
  if (p.T <= 4) return run<FMT, 4>(p, s);
  if (p.T <= 8) return run<FMT, 8>(p, s);
  return run<FMT, 16>(p, s);
}

// parts of K that y has room for: small batches only, where tasks are few
int k_split(const moe_config &c) { return c.num_tokens * c.top_k <= 32 ? MAX_KSPLIT : 1; }

struct FewLayout {
  size_t logits, xq, xs, xg, hg, h, h_lo, hs, hs_lo, rowmax, hq, y, total;
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
  const bool q4 = c.weight_dtype == MOE_Q4_AFFINE_G64, ints = i8 || q4;
  L.xq = take(ints ? (q4 ? 2 : 1) * T * d : 0);
  L.xs = take(ints ? sizeof(float) * T : 0);
  L.xg = take(q4 ? sizeof(float) * T * (d / 64) : 0);
  L.hg = take(q4 ? sizeof(float) * S * (F / 64) : 0);
  L.h = take((q4 ? sizeof(float) : 2) * S * F);
  L.h_lo = take(ints ? 0 : 2 * S * F);
  L.hs = take(2 * T * Fs);
  L.hs_lo = take(2 * T * Fs);
  L.rowmax = take(ints ? sizeof(unsigned) * S : 0);
  L.hq = take(ints ? (q4 ? 2 : 1) * S * F : 0);
  L.y = take(sizeof(float) * (S * k_split(c) + (Fs ? T : 0)) * d);
  L.total = off;
  return L;
}

}  // namespace

bool few_supported(const moe_config &c) { return c.num_tokens <= kFewTokens && c.act_dtype == MOE_BF16; }

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
  p.xg = reinterpret_cast<float *>(ws + L.xg);
  p.hg = reinterpret_cast<float *>(ws + L.hg);
  p.h = reinterpret_cast<uint16_t *>(ws + L.h);
  p.hf = reinterpret_cast<float *>(ws + L.h);
  p.h_lo = (L.h_lo - L.h) / 2;
  p.hs = reinterpret_cast<uint16_t *>(ws + L.hs);
  p.hs_lo = (L.hs_lo - L.hs) / 2;
  p.rowmax = reinterpret_cast<unsigned *>(ws + L.rowmax);
  p.hq = reinterpret_cast<int8_t *>(ws + L.hq);
  p.y = reinterpret_cast<float *>(ws + L.y);
  p.y_rows = c.num_tokens * c.top_k;
  p.ksplit = k_split(c);
  switch (c.weight_dtype) {
    case MOE_BF16: return run_t<BF16>(p, s);
    case MOE_I8_CHANNEL: return run_t<I8>(p, s);
    default: return run_t<Q4>(p, s);
  }
}

}  // namespace moe
