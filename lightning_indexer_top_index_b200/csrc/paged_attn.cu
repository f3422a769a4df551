// MQA attention of the last T tokens of each sequence over a paged cache
// (K = V = the full 512-wide row), over all rows or those of chosen blocks.
//
// Work.  A job is one query token and up to 64 of its heads; its rows are cut
// into chunks of 64.  The chunks of all jobs, in order, are dealt out evenly
// to one CTA per SM, so that ragged lengths, few long sequences and many short
// ones all fill the machine; a CTA may end one job and begin another, and a
// job may span CTAs.  A job that one CTA holds whole is written out by it; the
// others leave partial results (m, l, O) that the merge kernel joins.
//
// A CTA has 19 warps:
//   * the scout finds each chunk's pool rows (block list, page table) up to
//     four chunks ahead and says where a job begins and ends;
//   * eight loader warps, eight rows each, fetch the stored rows a chunk ahead
//     into registers, expand them to bf16 (exact: every E2M1 or E4M3 value
//     times a power of two is a bf16 value while it is in its range) and store them as the swizzled
//     K-major tile X[64 rows][512], two of which are in shared memory.  Rows
//     that are not attended to are stored as zeros.  They go by quarters of 128
//     dims, and S begins with the half of the dims that is in while the other
//     is expanded; a half is refilled once O is done with its dims.  So the
//     stages of a chunk, whose lengths add up to the CTA's pace, overlap;
//   * one warp issues S[head][row] = Q . X^T (M = 64, N = 64, K = 512) and
//     another, when the chunk's probabilities are there, O^T[d][head] +=
//     X^T . P^T (M = 128 four times, N = 64, K = 64), both on tcgen05 with fp32
//     accumulators in TMEM, two of S and one of O.  (Before the waits were as
//     cheap as below, one warp that polled for whichever was ready took 123 us
//     instead of 102 for 256 queries of 1024 rows, and S in two or four
//     accumulators, whose products need not wait for one another, 104.);
//   * eight softmax warps, one per 16 heads and half of the chunk's rows, read
//     S in the 16x256b shape, in which the 32 lanes of a warp share the 16 heads
//     of its TMEM quarter (8 head pairs x 4 column groups), so row maxima take
//     two shuffles and no lane idles.  The running maximum is only a
//     reference (p = 2^(s - m) may exceed 1), so it moves only when it rises
//     by more than 32 (base 2), and only then is the O so far rescaled in
//     TMEM: at 8 one of the 64 heads made most chunks pay for it.  Sums are of
//     the fp32 probabilities; floating point loses nothing by a common factor
//     up to 2^32.
//   P enters the second product as its bf16 value and the bf16 value of what
//   that rounding left, so it keeps 16 bits (2^-16 of each probability), as in
//   the attention over linear caches; both are products of the same rows.
//
// What bounds it.  For 256 queries of 1024 rows in E2M1 (84 us, 20 at the bf16
// rate of the matrix products) a CTA takes a chunk every 3500 cycles.  Its
// products (32 of 32 cycles, 32 of 48, both bound by their operands in shared
// memory) take 2560 of them; a loader warp, always busy, takes all of them for
// its 550 instructions, with 45 % of all issue slots used, 7800 instructions a
// chunk, a quarter of them in the expansion.  Sixteen loader warps of half as
// much each leave the others fewer slots and registers: 94 us.
//
// The loops are kept small (one place each for a product, a load, a store):
// unrolled over their chunks they outgrew the instruction cache, and the
// kernel spent half its time fetching code (a chunk took 8000 cycles).
#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "quant.cuh"
#include "tc.cuh"

namespace lidx {

namespace {

constexpr int kD = 512;
constexpr int kH = 64;                   // heads of a job
constexpr int kRows = 64;                // rows of a chunk
constexpr int kLoaders = 8;              // warps, eight rows each
constexpr int kSoftmaxWarps = 8;         // warp w: heads 16 (w % 4) .., rows 32 (w / 4) .. of a chunk
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoaders + 3);
constexpr int kIssueS = kSoftmaxWarps + kLoaders, kIssueO = kIssueS + 1, kScout = kIssueO + 1;  // their warps
constexpr int kRing = 4;                 // chunks the scout may be ahead
constexpr int kPanel = 64 * 128;         // one 64-line panel of X or Q: 64 dims
constexpr int kXBytes = 8 * kPanel;
constexpr int kQBytes = 8 * kPanel;
constexpr int kPHalf = kH * kRows * 2;   // P as bf16, then what its rounding left
constexpr int kPBytes = 2 * kPHalf;
constexpr uint32_t kOCol = 128;          // S of stage i at columns 64 i, O^T tile t at columns kOCol + 64 t
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 32.f;            // base-2 headroom of the reference maximum
constexpr int kMergeThreads = 256;
constexpr int kFew = 8, kSome = 32;      // partials that one warp joins, for 128 dims and for 32
constexpr int kBatch = 10;               // partials that a warp of the merge has in flight: two batches of 148 / 8
constexpr int kMergeCtas = 4;            // of the merge, for an SM
constexpr int kMaxCtas = 256;            // one CTA per SM

// What the scout says about a chunk.
constexpr uint32_t kFirst = 1u;  // the first chunk of its job in this CTA
constexpr uint32_t kLast = 2u;   // the last one
constexpr uint32_t kWhole = 4u;  // ... and the CTA holds all of the job's chunks
struct __align__(16) Chunk {
  int32_t row[kRows];  // pool rows; -1: not attended to
  uint32_t valid[2];   // bit r: row r is attended to
  int32_t job;
  uint32_t flags;
};

struct __align__(16) Smem {
  Chunk ring[kRing];
  uint64_t ring_full[kRing], ring_free[kRing];
  uint64_t q_full;
  uint64_t x_full[2][2];          // half of the dims of a stage's rows are in
  uint64_t x_free[2][2];          // the second product is done with half of its dims (with the second half: and with P)
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_free;                // the finished job's O has been read
  uint64_t drained[2];            // every S or O product issued is done (only after a wait gave up)
  uint32_t tmem_base;
  uint32_t abort;
  float alpha[kH];                // rescale factors of a chunk
  float top[2][kH];               // a chunk's maxima, by half of its rows
  float sums[2][kH];              // a job's sums, by half of the rows
  float l[kH];                    // 1 / sum
  // the CTA's first chunk
  int32_t job, chunk;
  int32_t scan[kThreads / 32];
};

constexpr size_t smem_bytes() { return kQBytes + 2 * kXBytes + 2 * kPBytes + sizeof(Smem); }
static_assert(smem_bytes() <= 227 * 1024, "a CTA's shared memory");

// A job that spans CTAs, written by the second of them: its chunks are
// [start, end) of all chunks (job -1: the CTA is no job's second one).
struct __align__(16) Split {
  int32_t job, start, end, total;
};

// Where the partial results and the split jobs lie in the workspace.
struct Scratch {
  uint32_t *status;
  Split *split;  // [G]
  float2 *ml;    // [2 * G][kH]: maximum, sum
  float4 *o;     // [2 * G][kH / 4][kD], four heads together: as TMEM holds them
};

// The job list.
struct Jobs {
  int32_t n;       // B * T * groups of heads
  int32_t group_shift;  // 0: one group of up to 64 heads, 1: two
  int32_t G;       // CTAs
};

// The chunks are dealt out in runs of base or base + 1 (the first `more` CTAs).
struct Deal {
  int32_t base, more;
  __device__ __forceinline__ Deal(int32_t total, int32_t G) : base(total / G), more(total % G) {}
  __device__ __forceinline__ int32_t start(int32_t g) const { return g * base + min(g, more); }  // CTA g's first chunk
  __device__ __forceinline__ int32_t owner(int32_t c) const {  // the CTA that holds chunk c
    const int32_t big = more * (base + 1);
    return c < big ? c / (base + 1) : more + (c - big) / max(base, 1);
  }
};

// Entries of job's row list: rows for the dense case, rows of the listed blocks otherwise.
__device__ __forceinline__ int32_t job_rows(const lidx_paged_attn_args &a, int32_t job, int gs, int shift) {
  const int32_t bt = job >> gs;
  if (a.blocks) return (a.n_sel ? min(max(fetch(a.n_sel + bt), 0), a.n_blocks) : a.n_blocks) << shift;
  bool cut;
  return max(cut_len(fetch(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T), 0);
}
__device__ __forceinline__ int32_t job_chunks(const lidx_paged_attn_args &a, int32_t job, int gs, int shift) {
  return (job_rows(a, job, gs, shift) + kRows - 1) / kRows;
}

__device__ __forceinline__ bool elect() {  // true in one lane of a converged warp, always the same
  uint32_t r;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " elect.sync _|p, 0xFFFFFFFF;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(r));
  return r != 0u;
}

// tc::mbar_wait for a whole warp: the same answer in all lanes.  Its loop is
// kept rolled, and the vote is in it, so that the warp stays together: with lane
// 0 waiting and a shuffle of its answer, each hand-over between the roles was a
// few hundred cycles longer (100 against 87 us for 256 queries of 1024 rows), with the lanes
// looping apart and a vote at the end 88.5.  Polling without the hardware's
// suspension (test_wait) takes issue slots from the others: 91.5.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile uint32_t *abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < tc::kWaitLimit; i++) {
    if (__all_sync(0xFFFFFFFFu, tc::mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xFFFFFFFFu, *abort)) return false;
  }
  *abort = 1u;
  return false;
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; 2^-inf = 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t bar_or(int id, int n, uint32_t v) {
  uint32_t r;
  asm volatile(
      "{\n"
      " .reg .pred p, q;\n"
      " setp.ne.u32 p, %3, 0;\n"
      " barrier.cta.red.or.pred q, %1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n"
      "}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(v)
      : "memory");
  return r;
}

// S of 16 heads x 32 rows: lane l holds heads l/4 (regs 4u, 4u+1) and l/4 + 8
// (regs 4u+2, 4u+3), rows 8u + 2 (l % 4) and the next.
__device__ __forceinline__ void tmem_ld_s(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 consecutive columns of this thread's lane, without waiting.
__device__ __forceinline__ void tmem_ld16_issue(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_pin16(uint32_t (&r)[16]) {  // no use of them before the wait above this
#pragma unroll
  for (int i = 0; i < 16; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; i++) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 64-head box of a [B * T][H][512] query tensor; heads beyond H read as zeros.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, uint64_t *bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A quarter (128 dims, two panels of X) of a row in 16-byte pieces as stored;
// a loader warp's eight rows of it are kIters pieces a lane.
template <int kFmt>
struct Fmt {
  static constexpr int kPieces = kFmt == LIDX_E2M1 ? 4 : kFmt == LIDX_E4M3 ? 8 : 16;
  static constexpr int kIters = kPieces / 4;
  static constexpr int kRowsPerIter = 32 / kPieces;
};

// Eight E4M3 codes times their block's scale (both halves of s) as bf16.
__device__ __forceinline__ uint4 expand_e4m3(uint32_t x, uint32_t y, uint32_t s) {
  return make_uint4(mul_bf16x2(e4m3x2_to_bf16x2(x), s), mul_bf16x2(e4m3x2_to_bf16x2(x >> 16), s),
                    mul_bf16x2(e4m3x2_to_bf16x2(y), s), mul_bf16x2(e4m3x2_to_bf16x2(y >> 16), s));
}

// Piece p of row r expanded to bf16 into the quarter's panels at x.  Lanes of
// the second panel take their 16-byte chunks in another order, so that the
// eight lanes that store together hit all banks.
template <int kFmt>
__device__ __forceinline__ void store_piece(uint8_t *x, int r, int p, const uint4 &v, uint32_t scale) {
  uint8_t *row = x + r * 128 + (p / (Fmt<kFmt>::kPieces / 2)) * kPanel;
  const int swz = r & 7;
  if constexpr (kFmt == LIDX_BF16) {
    *reinterpret_cast<uint4 *>(row + (((p & 7) ^ swz) << 4)) = v;
  } else if constexpr (kFmt == LIDX_E2M1) {
    const int turn = p & 2;
    const uint32_t w[4] = {turn ? v.z : v.x, turn ? v.w : v.y, turn ? v.x : v.z, turn ? v.y : v.w};
    const E2m1Scale s = E2m1Scale::of(scale);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint32_t o[4];
      s.expand(w[i], o);
      *reinterpret_cast<uint4 *>(row + (((4 * (p & 1) + (i ^ turn)) ^ swz) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    const int turn = (p >> 2) & 1;
    const uint32_t w[4] = {turn ? v.z : v.x, turn ? v.w : v.y, turn ? v.x : v.z, turn ? v.y : v.w};
    const uint32_t s = e8m0_to_bf16x2(scale);
#pragma unroll
    for (int i = 0; i < 2; i++)
      *reinterpret_cast<uint4 *>(row + (((2 * (p & 3) + (i ^ turn)) ^ swz) << 4)) = expand_e4m3(w[2 * i], w[2 * i + 1], s);
  }
}

// The same of a quarter with one panel of codes, in pieces of half the size.
template <int kFmt>
__device__ __forceinline__ void store_half_piece(uint8_t *x, int r, int p, const uint4 &v, uint32_t scale) {
  uint8_t *row = x + r * 128;
  const int swz = r & 7;
  if constexpr (kFmt == LIDX_E2M1) {
    const E2m1Scale s = E2m1Scale::of(scale);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint32_t o[4];
      s.expand(i ? v.y : v.x, o);
      *reinterpret_cast<uint4 *>(row + (((2 * p + i) ^ swz) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    *reinterpret_cast<uint4 *>(row + ((p ^ swz) << 4)) = expand_e4m3(v.x, v.y, e8m0_to_bf16x2(scale));
  }
}

// Pool row of entry e of a job's row list, or -1.
__device__ __forceinline__ int32_t entry_row(const lidx_paged_attn_args &a, int32_t bt, int shift, int32_t e,
                                             int32_t seen, int32_t n_list, bool &bounds) {
  if (e >= n_list) return -1;
  int32_t r = e, b = bt / a.T;
  if (a.blocks) {
    const int32_t j = fetch(a.blocks + static_cast<int64_t>(bt) * a.ld_blocks + (e >> shift));
    if (j < 0 || j >= a.cache.max_pages) {
      bounds |= j != -1;
      return -1;
    }
    r = (j << shift) | (e & (a.cache.page_rows - 1));
  }
  if (r >= seen) return -1;
  const int32_t p = pool_row(a.cache, shift, b, r);
  bounds |= p < 0;
  return p;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ lidx_paged_attn_args a,
                      const Jobs jobs, const int shift, const Scratch ws) {
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle wants panels at multiples of 1024
  uint8_t *sQ = smem;
  uint8_t *sX = sQ + kQBytes;      // stage i at sX + i * kXBytes
  uint8_t *sP = sX + 2 * kXBytes;  // stage i at sP + i * kPBytes
  Smem *sm = reinterpret_cast<Smem *>(sP + 2 * kPBytes);
  volatile uint32_t *abort_flag = &sm->abort;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // the same in all lanes, for the compiler to see
  const int gs = jobs.group_shift;

  if (tid == 0) {
    tc::mbar_init(&sm->q_full, 1);
#pragma unroll
    for (int i = 0; i < kRing; i++) {
      tc::mbar_init(&sm->ring_full[i], 1);
      tc::mbar_init(&sm->ring_free[i], kSoftmaxWarps + kLoaders + 2);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
      for (int h = 0; h < 2; h++) tc::mbar_init(&sm->x_full[i][h], kLoaders);
      tc::mbar_init(&sm->x_free[i][0], 1);
      tc::mbar_init(&sm->x_free[i][1], 1);
      tc::mbar_init(&sm->p_full[i], kSoftmaxWarps);
      tc::mbar_init(&sm->s_full[i], 1);
    }
    tc::mbar_init(&sm->o_free, kSoftmaxWarps);
    tc::mbar_init(&sm->drained[0], 1);
    tc::mbar_init(&sm->drained[1], 1);
    sm->abort = 0;
    tc::fence_barrier_init();
    tc::tma_prefetch_desc(&tm_q);
  }
  if (warp == 0) tc::tmem_alloc(&sm->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  pdl_trigger();
  pdl_wait();  // queries, lens, tables and rows may come from the previous kernel
  const uint32_t tmem = sm->tmem_base;

  // ---- the schedule: prefix sums of the jobs' chunks, this CTA's range of them
  int32_t total, my0, my1;
  {
    const int per = (jobs.n + kThreads - 1) / kThreads;
    const int j0 = min(tid * per, jobs.n), j1 = min(j0 + per, jobs.n);
    int32_t mine = 0;
#pragma unroll 1
    for (int j = j0; j < j1; j++) mine += job_chunks(a, j, gs, shift);
    const int32_t incl = warp_inclusive_scan(mine);
    if (lane == 31) sm->scan[warp] = incl;
    __syncthreads();
    int32_t before = incl - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
      const int32_t s = sm->scan[w];
      if (w < warp) before += s;
      total += s;
    }
    const Deal deal(total, jobs.G);
    my0 = deal.start(blockIdx.x);
    my1 = deal.start(blockIdx.x + 1);
    if (before <= my0 && my0 < before + mine) {
      int32_t at = before;
#pragma unroll 1
      for (int j = j0; j < j1; j++) {
        const int32_t m = job_chunks(a, j, gs, shift);
        if (at <= my0 && my0 < at + m) {
          sm->job = j;
          sm->chunk = my0 - at;
        }
        at += m;
      }
    }
    __syncthreads();
  }
  const int n = my1 - my0;  // this CTA's chunks
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return wait_all(bar, parity, abort_flag); };

  if (warp == kScout) {
    // -------------------------------------------------------------- scout
    int32_t job = 0, c = 0, left = 0, seen = 0, rows = 0;  // `left` chunks of the job from chunk c on
    bool bounds = false, whole = false;
    if (n > 0) {
      job = sm->job;
      c = sm->chunk;
    }
    const int32_t first_job = job, first_c = c;
    for (int i = 0; i < n; i++) {
      uint32_t flags = 0u;
      if (left == 0) {  // a job begins: the CTA's first, or the next one with rows
        if (i > 0) {
          job++;
          c = 0;
        }
        while ((rows = job_rows(a, job, gs, shift)) == 0) job++;
        left = (rows + kRows - 1) / kRows - c;
        const int32_t bt = job >> gs;
        bool cut;
        seen = cut_len(fetch(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T);
        bounds |= cut;
        whole = c == 0;
        flags = kFirst;
      }
      if (left == 1 || i + 1 == n) flags |= kLast | (whole && left == 1 ? kWhole : 0u);
      const int32_t bt = job >> gs;
      const int32_t p0 = entry_row(a, bt, shift, c * kRows + lane, seen, rows, bounds);
      const int32_t p1 = entry_row(a, bt, shift, c * kRows + 32 + lane, seen, rows, bounds);
      const uint32_t v0 = __ballot_sync(0xFFFFFFFFu, p0 >= 0), v1 = __ballot_sync(0xFFFFFFFFu, p1 >= 0);
      const int slot = i % kRing;
      if (i >= kRing && !warp_wait(&sm->ring_free[slot], (i / kRing - 1) & 1)) break;
      Chunk &k = sm->ring[slot];
      k.row[lane] = p0;
      k.row[lane + 32] = p1;
      if (lane == 0) {
        k.valid[0] = v0;
        k.valid[1] = v1;
        k.job = job;
        k.flags = flags;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->ring_full[slot]);
      c++;
      left--;
    }
    if (lane == 0) {  // does a job that began in the CTA before continue here, and is this its second CTA?
      Split sp;
      sp.job = -1;
      sp.start = my0 - first_c;
      sp.end = 0;
      sp.total = total;
      const Deal deal(total, jobs.G);
      if (first_c > 0 && deal.start(static_cast<int32_t>(blockIdx.x) - 1) <= sp.start) {
        sp.job = first_job;
        sp.end = sp.start + (job_rows(a, first_job, gs, shift) + kRows - 1) / kRows;
      }
      ws.split[blockIdx.x] = sp;
    }
    if (bounds) raise_status(ws.status, LIDX_DEV_BOUNDS);
  } else if (warp >= kSoftmaxWarps && warp < kIssueS) {
    // ------------------------------------------------------------ loaders
    using F = Fmt<kFmt>;
    constexpr bool kQuant = kFmt != LIDX_BF16;
    const lidx_kv &kv = a.cache.rows;
    const int from = 8 * (warp - kSoftmaxWarps);  // the warp's rows of a chunk
    const int piece = lane % F::kPieces;
    const uint8_t *data = static_cast<const uint8_t *>(kv.data) + piece * 16;
    const int64_t pitch = kFmt == LIDX_BF16 ? 2 * kv.ld : kv.ld;
    const uint8_t *scales = kv.scale + (kFmt == LIDX_E2M1 ? piece : piece / 4);
    const uint8_t *rope = static_cast<const uint8_t *>(kv.rope) + (lane % 8) * 16;
    // the last quarter has codes for its first panel only: the lanes take half as many of it
    const uint8_t *last_data = data + 3 * (F::kPieces * 16) - piece * 8;
    const uint8_t *last_scales = kv.scale + (kFmt == LIDX_E2M1 ? 12 + piece / 2 : 6);
    uint4 v[4][F::kIters], rv[2];
    uint32_t sc[4][F::kIters];
#pragma unroll 1
    for (int i = 0; i <= n; i++) {  // chunk i - 1 into shared memory, chunk i into registers, a quarter at a time
      int32_t row[F::kIters], rope_row[2];
      if (i < n) {
        const int slot = i % kRing;
        if (!warp_wait(&sm->ring_full[slot], (i / kRing) & 1)) break;
        const int32_t *rows = sm->ring[slot].row + from;
#pragma unroll
        for (int it = 0; it < F::kIters; it++) row[it] = rows[it * F::kRowsPerIter + lane / F::kPieces];
#pragma unroll
        for (int it = 0; it < 2; it++) rope_row[it] = rows[it * 4 + lane / 8];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->ring_free[slot]);
      }
      const int stage = (i - 1) & 1;
      bool ok = true;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        if (i > 0 && ok) {
          if (i > 2 && (q & 1) == 0) ok = warp_wait(&sm->x_free[stage][q >> 1], (((i - 1) >> 1) - 1) & 1);
          if (!ok) break;
          uint8_t *x = sX + stage * kXBytes + 2 * q * kPanel;
#pragma unroll
          for (int it = 0; it < F::kIters; it++) {
            const int r = from + it * F::kRowsPerIter + lane / F::kPieces;
            if (kQuant && q == 3) store_half_piece<kFmt>(x, r, piece, v[q][it], sc[q][it]);
            else store_piece<kFmt>(x, r, piece, v[q][it], sc[q][it]);
          }
          if (kQuant && q == 3) {
#pragma unroll
            for (int it = 0; it < 2; it++)
              store_piece<LIDX_BF16>(x + kPanel, from + it * 4 + lane / 8, lane % 8, rv[it], 0u);
          }
          if (q & 1) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm->x_full[stage][q >> 1]);
          }
        }
        if (i < n) {
#pragma unroll
          for (int it = 0; it < F::kIters; it++) {
            v[q][it] = make_uint4(0, 0, 0, 0);
            sc[q][it] = 127u;
            if (row[it] >= 0 && kQuant && q == 3) {
              const uint2 h = fetch(reinterpret_cast<const uint2 *>(last_data + row[it] * pitch));
              v[q][it].x = h.x;
              v[q][it].y = h.y;
              sc[q][it] = fetch(last_scales + row[it] * kv.ld_scale);
            } else if (row[it] >= 0) {
              v[q][it] = fetch(reinterpret_cast<const uint4 *>(data + row[it] * pitch + q * (F::kPieces * 16)));
              if (kQuant) sc[q][it] = fetch(scales + row[it] * kv.ld_scale + q * (kFmt == LIDX_E2M1 ? 4 : 2));
            }
          }
          if (kQuant && q == 3) {
#pragma unroll
            for (int it = 0; it < 2; it++) {
              rv[it] = make_uint4(0, 0, 0, 0);
              if (rope_row[it] >= 0) rv[it] = fetch(reinterpret_cast<const uint4 *>(rope + rope_row[it] * (2 * kv.ld_rope)));
            }
          }
        }
      }
      if (!ok) break;
    }
  } else if (warp == kIssueS) {
    // ------------------------------------------------- S = Q . X^T
    // The whole warp goes through the loop, so that descriptors and flags stay
    // in uniform registers, and one elected lane issues: with a single lane in
    // the loop each product took 100 cycles to issue, whatever its shape.
    const uint32_t idesc = tc::idesc_bf16(64, 64);
    const uint64_t q_desc = tc::desc_kmajor_sw128(tc::smem_u32(sQ));
    const uint64_t x_desc = tc::desc_kmajor_sw128(tc::smem_u32(sX));
    int begun = 0;  // jobs
    bool ok = true, q_there = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; i++) {
      const int slot = i % kRing;
      ok = wait_all(&sm->ring_full[slot], (i / kRing) & 1, abort_flag);
      if (!ok) break;
      if (sm->ring[slot].flags & kFirst) {  // a new job's Q, when the last one has been read for the last time
        if (i > 0) ok = wait_all(&sm->s_full[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag);
        if (!ok) break;
        const int32_t job = sm->ring[slot].job;
        if (elect()) {
          tc::mbar_arrive_expect_tx(&sm->q_full, kQBytes);
#pragma unroll 1
          for (int p = 0; p < 8; p++)
            tma_load_3d(sQ + p * kPanel, &tm_q, &sm->q_full, 64 * p, (job & ((1 << gs) - 1)) * kH, job >> gs);
        }
        __syncwarp();
        begun++;
        q_there = false;
      }
      if (!q_there) {
        q_there = wait_all(&sm->q_full, (begun - 1) & 1, abort_flag);
        ok = ok && q_there;
      }
#pragma unroll 1
      for (int h = 0; h < 2 && ok; h++) {  // as the halves of the rows come in
        ok = wait_all(&sm->x_full[i & 1][h], (i >> 1) & 1, abort_flag);
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t qd = q_desc + 4 * h * (kPanel >> 4), xd = x_desc + (i & 1) * (kXBytes >> 4) + 4 * h * (kPanel >> 4);
        if (elect()) {
#pragma unroll
          for (int j = 0; j < 16; j++) {  // panel j / 4, 32 bytes (j % 4) into it
            const uint32_t off = (j >> 2) * (kPanel >> 4) + (j & 3) * 2;
            tc::mma_bf16(tmem + 64 * (i & 1), qd + off, xd + off, idesc, h > 0 || j > 0);
          }
          if (h == 1) {
            tc::mbar_arrive(&sm->ring_free[slot]);
            tc::mma_commit(&sm->s_full[i & 1]);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) {  // a wait gave up: the copies and products in flight end before the CTA does
      volatile uint32_t unused = 0;
      if (!q_there) wait_all(&sm->q_full, (begun - 1) & 1, &unused);
      if (elect()) tc::mma_commit(&sm->drained[0]);
      __syncwarp();
      wait_all(&sm->drained[0], 0, &unused);
    }
  } else if (warp == kIssueO) {
    // ------------------------------------------------- O^T += X^T . P^T, by a warp of its own: neither product waits for the other's turn
    const uint32_t idesc = tc::idesc_bf16(128, 64, true, false);
    const uint64_t x_desc = tc::desc_mnmajor_sw128(tc::smem_u32(sX), kPanel, 1024);
    const uint64_t p_desc = tc::desc_kmajor_sw128(tc::smem_u32(sP));
    int begun = 0;  // jobs
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n && ok; i++) {
      const int slot = i % kRing;
      ok = wait_all(&sm->ring_full[slot], (i / kRing) & 1, abort_flag);
      if (!ok) break;
      const bool first = sm->ring[slot].flags & kFirst;
      __syncwarp();
      if (elect()) tc::mbar_arrive(&sm->ring_free[slot]);
      if (first) {
        if (begun > 0) ok = wait_all(&sm->o_free, (begun - 1) & 1, abort_flag);
        begun++;
      }
      ok = ok && wait_all(&sm->p_full[i & 1], (i >> 1) & 1, abort_flag);
      if (!ok) break;
      tc::tc_fence_after();
      const uint64_t xd = x_desc + (i & 1) * (kXBytes >> 4), pd = p_desc + (i & 1) * (kPBytes >> 4);
      if (elect()) {
        // two dim tiles at a time: the loaders may then refill their panels
#pragma unroll
        for (int dt = 0; dt < 4; dt += 2) {
#pragma unroll
          for (int kk = 0; kk < kRows / 16; kk++) {
#pragma unroll
            for (int k = dt; k < dt + 2; k++) {
              const uint64_t x = xd + ((2 * k * kPanel + kk * 2048) >> 4);
              tc::mma_bf16(tmem + kOCol + 64 * k, x, pd + kk * 2, idesc, !first || kk > 0);
              tc::mma_bf16(tmem + kOCol + 64 * k, x, pd + kk * 2 + (kPHalf >> 4), idesc, true);
            }
          }
          tc::mma_commit(&sm->x_free[i & 1][dt / 2]);
        }
      }
      __syncwarp();
    }
    if (!ok) {
      volatile uint32_t unused = 0;
      if (elect()) tc::mma_commit(&sm->drained[1]);
      __syncwarp();
      wait_all(&sm->drained[1], 0, &unused);
    }
  } else {
    // ------------------------------------------------------------ softmax
    // first, while the first rows are on their way: the jobs without rows, dealt out to the CTAs
#pragma unroll 1
    for (int32_t j = blockIdx.x; j < jobs.n; j += jobs.G) {
      if (job_rows(a, j, gs, shift) > 0) continue;
      const int32_t bt = j >> gs, g = j & ((1 << gs) - 1), heads = min(kH, a.H - g * kH);
      const int64_t row = static_cast<int64_t>(bt) * a.H + g * kH;
      uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * kD);
#pragma unroll 1
      for (int i = tid; i < heads * kD / 8; i += 32 * kSoftmaxWarps) o[i] = make_uint4(0, 0, 0, 0);
      if (a.lse && tid < heads) a.lse[row + tid] = -INFINITY;
      bool cut;
      cut_len(fetch(a.len + bt / a.T), a.cache, cut);
      if (cut && tid == 0) raise_status(ws.status, LIDX_DEV_BOUNDS);
    }
    const int half = warp >> 2, h0 = (warp & 3) * 16 + (lane >> 2), h1 = h0 + 8;  // this lane's heads
    // logits are s * c2 in base 2, c2 > 0: with a negative scale s changes sign instead, and with a
    // zero one it becomes zero (rows that are not attended to have -inf, and 0 * -inf would be NaN)
    const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
    const float c2 = sign == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // the reference maximum is the same in both halves; the sums are of this half's rows
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool first_segment = true;  // the CTA's first job
    bool fresh = true;          // nothing of the job is in O yet
    uint32_t next_valid = 0u, next_flags = 0u;  // what the scout says about the next chunk
    int32_t next_job = 0;
    // After a wait that gave up the warp touches neither TMEM nor global memory, and at the next
    // chunk's vote all eight leave together, so that none waits for another at a barrier.
    bool ok = true;
    auto look_ahead = [&](int i) {
      if (i >= n) return;
      const int slot = i % kRing;
      ok = warp_wait(&sm->ring_full[slot], (i / kRing) & 1) && ok;
      next_valid = sm->ring[slot].valid[half];
      next_job = sm->ring[slot].job;
      next_flags = ok ? sm->ring[slot].flags : 0u;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->ring_free[slot]);
    };
    look_ahead(0);
#pragma unroll 1
    for (int i = 0; i < n; i++) {
      const int stage = i & 1;
      const uint32_t valid = next_valid, flags = next_flags;
      const int32_t job = next_job;
      ok = warp_wait(&sm->s_full[stage], (i >> 1) & 1) && ok;
      float s0[8], s1[8];
      if (ok) {
        tc::tc_fence_after();
        uint32_t x[16];
        tmem_ld_s(tmem + quarter + 64 * stage + 32 * half, x);
        tc::tmem_ld_wait();
        tmem_pin16(x);
        tc::tc_fence_before();
#pragma unroll
        for (int u = 0; u < 8; u++) {  // row 8 (u / 2) + 2 (lane % 4) + u % 2 of the half
          const int k = 4 * (u >> 1) + (u & 1);
          s0[u] = __uint_as_float(x[k]);
          s1[u] = __uint_as_float(x[k + 2]);
        }
      }
      if (sign != 1.f || valid != 0xFFFFFFFFu) {
        const uint32_t bits = valid >> (2 * (lane & 3));
#pragma unroll
        for (int u = 0; u < 8; u++) {
          const bool in = (bits >> (8 * (u >> 1) + (u & 1))) & 1u;
          s0[u] = in ? s0[u] * sign : -INFINITY;
          s1[u] = in ? s1[u] * sign : -INFINITY;
        }
      }
      float t0 = s0[0], t1 = s1[0];
#pragma unroll
      for (int u = 1; u < 8; u++) {
        t0 = fmaxf(t0, s0[u]);
        t1 = fmaxf(t1, s1[u]);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, o));
        t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, o));
      }
      t0 *= c2;
      t1 *= c2;
      // the reference maximum moves only on rises above kLazy, in any head or half
      if (bar_or(1, 32 * kSoftmaxWarps, !ok || fresh || t0 > m0 + kLazy || t1 > m1 + kLazy)) {
        if ((lane & 3) == 0) {
          sm->top[half][h0] = t0;
          sm->top[half][h1] = t1;
        }
        if (bar_or(1, 32 * kSoftmaxWarps, !ok)) break;
        t0 = fmaxf(t0, sm->top[half ^ 1][h0]);
        t1 = fmaxf(t1, sm->top[half ^ 1][h1]);
        const float n0 = t0 <= m0 + kLazy ? m0 : fmaxf(t0, m0), n1 = t1 <= m1 + kLazy ? m1 : fmaxf(t1, m1);
        // (the first rise from -inf finds sums and an O of zeros)
        const float a0 = n0 == m0 || m0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
        const float a1 = n1 == m1 || m1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= a0;
        l1 *= a1;
        if (!fresh) {  // rescale O^T (lane = dim, columns = heads), when the last second product is done
          if (half == 0 && (lane & 3) == 0) {
            sm->alpha[h0] = a0;
            sm->alpha[h1] = a1;
          }
          bar_or(1, 32 * kSoftmaxWarps, 0u);
          ok = warp_wait(&sm->x_free[stage ^ 1][1], ((i - 1) >> 1) & 1) && ok;
          if (ok) {
            tc::tc_fence_after();
#pragma unroll 1
            for (int q = half; q < 16; q += 2) {
              const uint32_t ta = tmem + quarter + kOCol + 16 * q;
              float v[16];
              tc::tmem_ld16(ta, v);
#pragma unroll
              for (int h = 0; h < 16; h++) v[h] *= sm->alpha[16 * (q & 3) + h];
              tmem_st16(ta, v);
            }
            tmem_st_wait();
          }
        }
      }
      fresh = false;
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      // P^T line `head`: 16-byte pieces of eight rows, swizzled with head & 7.  (The stage's P and S are
      // free: this chunk's rows could only be stored when the product that read P(i - 2) was done.)
      uint8_t *p0 = sP + stage * kPBytes + h0 * 128 + 4 * (lane & 3), *p1 = p0 + 8 * 128;
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const float x0 = exp2_approx(fmaf(s0[2 * u], c2, -b0)), x1 = exp2_approx(fmaf(s0[2 * u + 1], c2, -b0));
        const float y0 = exp2_approx(fmaf(s1[2 * u], c2, -b1)), y1 = exp2_approx(fmaf(s1[2 * u + 1], c2, -b1));
        l0 += x0 + x1;
        l1 += y0 + y1;
        const __nv_bfloat162 px = __floats2bfloat162_rn(x0, x1), py = __floats2bfloat162_rn(y0, y1);
        const uint32_t wx = *reinterpret_cast<const uint32_t *>(&px), wy = *reinterpret_cast<const uint32_t *>(&py);
        const __nv_bfloat162 qx = __floats2bfloat162_rn(x0 - bf16x2_lo(wx), x1 - bf16x2_hi(wx));
        const __nv_bfloat162 qy = __floats2bfloat162_rn(y0 - bf16x2_lo(wy), y1 - bf16x2_hi(wy));
        const int at = ((4 * half + u) ^ (h0 & 7)) << 4;
        *reinterpret_cast<uint32_t *>(p0 + at) = wx;
        *reinterpret_cast<uint32_t *>(p1 + at) = wy;
        *reinterpret_cast<uint32_t *>(p0 + kPHalf + at) = *reinterpret_cast<const uint32_t *>(&qx);
        *reinterpret_cast<uint32_t *>(p1 + kPHalf + at) = *reinterpret_cast<const uint32_t *>(&qy);
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->p_full[stage]);
      look_ahead(i + 1);

      if (flags & kLast) {  // this CTA's part of the job is done
        const int32_t bt = job >> gs, g = job & ((1 << gs) - 1);
        const bool out_now = flags & kWhole;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
          l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
        }
        const int h = (lane & 1) ? h1 : h0;  // lanes with lane % 4 < 2 look after a head each
        float l = (lane & 1) ? l1 : l0;
        const float m = (lane & 1) ? m1 : m0;
        if ((lane & 3) < 2) sm->sums[half][h] = l;
        bar_or(1, 32 * kSoftmaxWarps, 0u);
        const int heads = min(kH, a.H - g * kH);
        const int64_t out_row = static_cast<int64_t>(bt) * a.H + g * kH;
        const int64_t slot_o = 2 * static_cast<int64_t>(blockIdx.x) + (first_segment ? 0 : 1);
        if ((lane & 3) < 2 && half == 0 && ok) {
          l += sm->sums[1][h];
          if (out_now) {
            sm->l[h] = l == 0.f ? 0.f : 1.f / l;
            if (a.lse && h < heads) a.lse[out_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            ws.ml[slot_o * kH + h] = make_float2(m, l);
          }
        }
        bar_or(1, 32 * kSoftmaxWarps, 0u);  // sm->l is in
        ok = warp_wait(&sm->x_free[stage][1], (i >> 1) & 1) && ok;
        if (ok) {
          tc::tc_fence_after();
          uint32_t next[16];
          tmem_ld16_issue(tmem + quarter + kOCol + 16 * half, next);
#pragma unroll 1
          for (int q = half; q < 16; q += 2) {  // 16 heads of a dim tile at a time, the next ones on their way
            const int d = 128 * (q >> 2) + 32 * (warp & 3) + lane, hb = 16 * (q & 3);
            float v[16];
            tc::tmem_ld_wait();
            tmem_pin16(next);
#pragma unroll
            for (int k = 0; k < 16; k++) v[k] = __uint_as_float(next[k]);
            if (q + 2 < 16) tmem_ld16_issue(tmem + quarter + kOCol + 16 * (q + 2), next);
            if (out_now) {
              // Lane = dim, registers = heads.  Two lanes swap halves, the even one's for the odd heads, so
              // that each has two dims of every other head: a store writes 64 bytes of two heads.
              const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;  // odd: other's high, own high half; even: own low, other's low
              uint32_t *o = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + (out_row + hb + (lane & 1)) * kD + (d & ~1));
#pragma unroll
              for (int k = 0; k < 8; k++) {
                const float2 l2 = *reinterpret_cast<const float2 *>(&sm->l[hb + 2 * k]);
                const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * k] * l2.x, v[2 * k + 1] * l2.y);
                const uint32_t own = *reinterpret_cast<const uint32_t *>(&two);
                const uint32_t w = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), pick);
                if (hb + 2 * k + (lane & 1) < heads) o[k * kD] = w;
              }
            } else {
              float4 *o = ws.o + (slot_o * (kH / 4) + hb / 4) * kD + d;
#pragma unroll
              for (int k = 0; k < 4; k++) o[k * kD] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          }
          tc::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->o_free);
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        first_segment = false;
        fresh = true;
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && sm->abort) raise_status(ws.status, LIDX_DEV_TIMEOUT);
}

// A partial's weight and its part of the sum, given the joint maximum M.
__device__ __forceinline__ float weight_of(float m, float M) { return m == M ? 1.f : exp2_approx(m - M); }

// Joins the partial results of jobs that span CTAs.  An item is such a job,
// four of its heads and 32 or 128 of its dims (lane = dim).  First the partials'
// weights are found, a lane or a thread for each partial, then the weighted sum
// runs over the partials, in their order.  Where a job has up to 32 of them, as
// with many short jobs, a warp joins an item by itself; where it has more, the
// eight warps of the CTA take every eighth partial each and their sums meet in
// shared memory (8 sequences of 15000 rows, 19 partials a job: 61 us so, 48 by a
// warp).  It is bound by the latency of a few dependent reads of L2, so what
// helps is many of them in flight (112 registers): held to 80 registers for a
// third CTA on the SM it took 1 to 2 us more.
__global__ void __launch_bounds__(kMergeThreads, 2) paged_attn_merge_kernel(const lidx_paged_attn_args a, const Jobs jobs,
                                                                         const Scratch ws) {
  constexpr int kWarps = kMergeThreads / 32, kItems = (kH / 4) * (kD / 32);
  __shared__ Split list[3][kMaxCtas];  // jobs with few, some and many partials
  __shared__ int32_t count[3][kWarps];
  __shared__ float4 weight_s[kMaxCtas], acc_s[kWarps][32], red_s[2][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();  // the partial results come from the previous kernel
  // the split jobs, in the same order in every CTA (kMaxCtas <= kMergeThreads)
  Split sp;
  sp.job = -1;
  if (tid < jobs.G) sp = ws.split[tid];
  int kind = -1;
  if (sp.job >= 0) {
    const Deal deal(sp.total, jobs.G);
    const int n = deal.owner(sp.end - 1) - deal.owner(sp.start) + 1;
    kind = n <= kFew ? 0 : n <= kSome ? 1 : 2;
  }
  int n_of[3], at = 0;
#pragma unroll
  for (int c = 0; c < 3; c++) {
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, kind == c);
    if (lane == 0) count[c][warp] = __popc(mask);
    if (kind == c) at = __popc(mask & ((1u << lane) - 1u));
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 3; c++) {
    n_of[c] = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      if (w < warp && kind == c) at += count[c][w];
      n_of[c] += count[c][w];
    }
  }
  if (kind >= 0) list[kind][at] = sp;
  __syncthreads();

  float m[4], l[4], e[4];  // of four heads of the partial that the thread looks after
  auto look = [&](const float2 *ml) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float2 x = ml ? ml[k] : make_float2(-INFINITY, 0.f);
      m[k] = x.x;
      l[k] = x.y;
    }
  };
  // the job is the CTA's first one unless the CTA began with an earlier job
  auto slot_of = [&](const Deal &deal, int32_t c, int32_t start) { return 2 * c + (deal.start(c) < start ? 1 : 0); };
  auto write = [&](const Split &sj, int h, int d0, float M, float L, float A) {  // head h of the job's group
    const int32_t bt = sj.job >> jobs.group_shift, group = sj.job & ((1 << jobs.group_shift) - 1);
    if (group * kH + h >= a.H) return;
    const int64_t row = static_cast<int64_t>(bt) * a.H + group * kH + h;
    static_cast<__nv_bfloat16 *>(a.out)[row * kD + d0 + lane] = __float2bfloat16_rn(A * (L == 0.f ? 0.f : 1.f / L));
    if (a.lse && d0 == 0 && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  };

  // by a warp: kLanes >= the partials, kJ * 32 dims
  auto join = [&](const Split *jobs_of, int n_jobs, auto lanes_c, auto j_c) {
    constexpr int kLanes = decltype(lanes_c)::value, kJ = decltype(j_c)::value, kPer = kItems / kJ;
#pragma unroll 1
    for (int item = blockIdx.x * kWarps + warp; item < n_jobs * kPer; item += gridDim.x * kWarps) {
      const Split sj = jobs_of[item / kPer];
      constexpr int kSlices = kD / (32 * kJ);
      const int h4 = (item % kPer) / kSlices, d0 = 32 * kJ * (item % kSlices);
      const Deal deal(sj.total, jobs.G);
      const int32_t from = deal.owner(sj.start), n = deal.owner(sj.end - 1) - from + 1;
      const int part = lane % kLanes;  // the lane's partial
      look(part < n ? ws.ml + slot_of(deal, from + part, sj.start) * kH + 4 * h4 : nullptr);
      float M[4], L[4], A[4][kJ] = {};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        M[k] = m[k];
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) M[k] = fmaxf(M[k], __shfl_xor_sync(0xFFFFFFFFu, M[k], o));
        e[k] = part < n ? weight_of(m[k], M[k]) : 0.f;
        L[k] = e[k] * l[k];
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) L[k] += __shfl_xor_sync(0xFFFFFFFFu, L[k], o);
      }
#pragma unroll (8 / kJ)
      for (int c = 0; c < n; c++) {
        const float4 *o = ws.o + static_cast<size_t>(slot_of(deal, from + c, sj.start) * (kH / 4) + h4) * kD + d0 + lane;
        float4 v[kJ];
#pragma unroll
        for (int j = 0; j < kJ; j++) v[j] = o[32 * j];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float w = __shfl_sync(0xFFFFFFFFu, e[k], c);
#pragma unroll
          for (int j = 0; j < kJ; j++) A[k][j] = fmaf(w, reinterpret_cast<const float *>(&v[j])[k], A[k][j]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; k++)
#pragma unroll
        for (int j = 0; j < kJ; j++) write(sj, 4 * h4 + k, d0 + 32 * j, M[k], L[k], A[k][j]);
    }
  };
  join(list[0], n_of[0], std::integral_constant<int, kFew>(), std::integral_constant<int, 4>());
  join(list[1], n_of[1], std::integral_constant<int, kSome>(), std::integral_constant<int, 1>());

#pragma unroll 1
  for (int item = blockIdx.x; item < n_of[2] * kItems; item += gridDim.x) {
    const Split sj = list[2][item / kItems];
    const int h4 = (item % kItems) / (kD / 32), d0 = 32 * (item % (kD / 32));
    const Deal deal(sj.total, jobs.G);
    const int32_t from = deal.owner(sj.start), n = deal.owner(sj.end - 1) - from + 1;  // <= kMaxCtas
    look(tid < n ? ws.ml + slot_of(deal, from + tid, sj.start) * kH + 4 * h4 : nullptr);
    float M[4], L[4];
#pragma unroll
    for (int k = 0; k < 4; k++) M[k] = warp_max(m[k]);
    if (lane == 0) red_s[0][warp] = make_float4(M[0], M[1], M[2], M[3]);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; w++)
#pragma unroll
      for (int k = 0; k < 4; k++) M[k] = fmaxf(M[k], reinterpret_cast<const float *>(&red_s[0][w])[k]);
#pragma unroll
    for (int k = 0; k < 4; k++) {
      e[k] = tid < n ? weight_of(m[k], M[k]) : 0.f;
      L[k] = warp_sum(tid < n ? e[k] * l[k] : 0.f);
    }
    if (tid < n) weight_s[tid] = make_float4(e[0], e[1], e[2], e[3]);
    if (lane == 0) red_s[1][warp] = make_float4(L[0], L[1], L[2], L[3]);
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int32_t c0 = warp; c0 < n; c0 += kBatch * kWarps) {
      float4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const int32_t c = c0 + u * kWarps;
        v[u] = c < n ? ws.o[static_cast<size_t>(slot_of(deal, from + c, sj.start) * (kH / 4) + h4) * kD + d0 + lane]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kBatch; u++) {
        const float4 w = weight_s[min(c0 + u * kWarps, kMaxCtas - 1)];
        const bool in = c0 + u * kWarps < n;
        acc.x = fmaf(in ? w.x : 0.f, v[u].x, acc.x);
        acc.y = fmaf(in ? w.y : 0.f, v[u].y, acc.y);
        acc.z = fmaf(in ? w.z : 0.f, v[u].z, acc.z);
        acc.w = fmaf(in ? w.w : 0.f, v[u].w, acc.w);
      }
    }
    acc_s[warp][lane] = acc;
    __syncthreads();
    if (warp < 4) {  // warp k finishes head k
      float A = 0.f, Ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        A += reinterpret_cast<const float *>(&acc_s[w][lane])[warp];
        Ls += reinterpret_cast<const float *>(&red_s[1][w])[warp];
      }
      write(sj, 4 * h4 + warp, d0, warp == 0 ? M[0] : warp == 1 ? M[1] : warp == 2 ? M[2] : M[3], Ls, A);
    }
    __syncthreads();
  }
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

int64_t most_chunks(const lidx_paged_attn_args &a) {  // of a job
  const int64_t rows = static_cast<int64_t>(a.blocks ? a.n_blocks : a.cache.max_pages) * a.cache.page_rows;
  return (rows + kRows - 1) / kRows;
}

int64_t job_count(const lidx_paged_attn_args &a) { return static_cast<int64_t>(a.B) * a.T * ((a.H + kH - 1) / kH); }

Jobs plan(const lidx_paged_attn_args &a) {
  Jobs j;
  j.group_shift = a.H > kH ? 1 : 0;
  j.n = static_cast<int32_t>(job_count(a));
  j.G = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(std::min(sm_count(), kMaxCtas), job_count(a) * most_chunks(a))));
  return j;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

template <int kFmt>
cudaError_t launch(const CUtensorMap &tm, const lidx_paged_attn_args &a, const Jobs &j, const Scratch &s, cudaStream_t st) {
  const size_t smem = smem_bytes();
  cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<kFmt>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_attn_kernel<kFmt>, dim3(j.G), dim3(kThreads), smem, st, (a.flags & LIDX_LAUNCH_PDL) != 0,
                       tm, a, j, page_shift(a.cache), s);
}

}  // namespace

bool paged_attn_supported(const lidx_paged_attn_args &a) {
  const int64_t rows = static_cast<int64_t>(a.blocks ? a.n_blocks : a.cache.max_pages) * a.cache.page_rows;
  // entries of a job are counted in 32 bits up to the end of its last chunk
  return rows <= INT32_MAX - (kRows - 1) && job_count(a) <= (1 << 24) && job_count(a) * most_chunks(a) <= INT32_MAX;
}

size_t paged_attn_workspace(const lidx_paged_attn_args &a) {
  const Jobs j = plan(a);
  return LIDX_WS_HEADER + align256(j.G * sizeof(Split)) + static_cast<size_t>(j.G) * 2 * kH * (sizeof(float2) + kD * 4);
}

int paged_attn_launches(const lidx_paged_attn_args &) { return 2; }  // the attention and the merge

cudaError_t launch_paged_attn(const lidx_paged_attn_args &a, void *ws, cudaStream_t st) {
  const Jobs j = plan(a);
  Scratch s;
  char *p = static_cast<char *>(ws);
  s.status = reinterpret_cast<uint32_t *>(p);
  p += LIDX_WS_HEADER;
  s.split = reinterpret_cast<Split *>(p);
  p += align256(j.G * sizeof(Split));
  s.ml = reinterpret_cast<float2 *>(p);
  p += static_cast<size_t>(j.G) * 2 * kH * sizeof(float2);
  s.o = reinterpret_cast<float4 *>(p);
  CUtensorMap tm;
  if (!make_tmap_3d(&tm, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kD, a.H, static_cast<uint64_t>(a.B) * a.T, 64, kH,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e;
  switch (a.cache.rows.dtype) {
    case LIDX_E2M1: e = launch<LIDX_E2M1>(tm, a, j, s, st); break;
    case LIDX_E4M3: e = launch<LIDX_E4M3>(tm, a, j, s, st); break;
    default: e = launch<LIDX_BF16>(tm, a, j, s, st); break;
  }
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_attn_merge_kernel, dim3(kMergeCtas * sm_count()), dim3(kMergeThreads), 0, st, true, a, j, s);
}

}  // namespace lidx
