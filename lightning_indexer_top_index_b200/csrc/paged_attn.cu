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
// A CTA has 14 warps:
//   * the scout finds each chunk's pool rows (block list, page table) up to
//     four chunks ahead and says where a job begins and ends;
//   * eight loader warps, one per 64-dim slab of the row, fetch the stored
//     rows a chunk ahead into registers, expand them to bf16 (exact: every
//     E2M1 or E4M3 value times a power of two is a bf16 value) and store them
//     as the swizzled K-major tile X[64 rows][512], two of which are in shared
//     memory.  Rows that are not attended to are stored as zeros;
//   * one thread issues S[head][row] = Q . X^T (M = 64, N = 64, K = 512) and,
//     when the chunk's probabilities are there, O^T[d][head] += X^T . P^T
//     (M = 128 four times, N = 64, K = 64), both on tcgen05 with fp32
//     accumulators in TMEM.  Products that add to the same accumulator wait
//     for one another, so S is summed in four parts (K quarters) and O's four
//     dim tiles are taken in turn;
//   * four softmax warps read S in the 16x256b shape, in which the 32 lanes of
//     a warp share the 16 heads of its TMEM quarter (8 head pairs x 4 column
//     groups), so row maxima take two shuffles and no lane idles.  S is free
//     for the next chunk as soon as it is read.  The running maximum is only a
//     reference (p = 2^(s - m) may exceed 1), so it moves only when it rises
//     by more than 32 (base 2), and only then is the O so far rescaled in
//     TMEM: at 8 one of the 64 heads made most chunks pay for it.  Sums are of
//     the fp32 probabilities; floating point loses nothing by a common factor
//     up to 2^32.
//   P is rounded to bf16 for the second product, 2^-9 of each probability.  O
//   is divided by the sum of the rounded ones, so that its weights add up to
//   one and a row that has nearly all of it comes out exactly (by the unrounded
//   sum the error over peaked rows was 1.6 times that of an exact P); lse takes
//   the unrounded sum.
//
// The loops are kept small (one place each for a product, a load, a store):
// unrolled over their chunks they outgrew the instruction cache, and the
// kernel spent half its time fetching code (a chunk took 8000 cycles).
#include <algorithm>

#include "paged.cuh"
#include "quant.cuh"
#include "tc.cuh"

namespace lidx {

namespace {

constexpr int kD = 512;
constexpr int kH = 64;                   // heads of a job
constexpr int kRows = 64;                // rows of a chunk
constexpr int kLoaders = 8;              // warps; warp i of them fills dims [64 i, 64 i + 64)
constexpr int kSoftmaxWarps = 4;
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoaders + 2);
constexpr int kMma = kSoftmaxWarps + kLoaders, kScout = kMma + 1;  // their warps
constexpr int kRing = 4;                 // chunks the scout may be ahead
constexpr int kPanel = 64 * 128;         // one 64-line panel of X or Q: 64 dims
constexpr int kXBytes = 8 * kPanel;
constexpr int kQBytes = 8 * kPanel;
constexpr int kPBytes = kH * kRows * 2;
constexpr int kParts = 4;                // partial sums of S, at columns 64 i
constexpr uint32_t kOCol = 64 * kParts;  // O^T tile t at columns kOCol + 64 t
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 32.f;            // base-2 headroom of the reference maximum
constexpr int kMergeThreads = 256;
constexpr int kFew = 8;                  // partials that one warp joins
constexpr int kMaxCtas = 256;            // one CTA per SM
constexpr uint32_t kIdleLimit = 1u << 24;  // rounds without work after which the issuing warp gives up (seconds)

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
  uint64_t x_full[2], x_free[2];  // a stage's rows are in / its second product is done (X and P free again)
  uint64_t s_full, s_free;
  uint64_t p_full[2];
  uint64_t o_free;                // the finished job's O has been read
  uint64_t drained;               // every product issued is done (only after a wait gave up)
  uint32_t tmem_base;
  uint32_t abort;
  float alpha[2][kH];             // rescale factors of a chunk
  float l[kH];                    // 1 / sum of the rounded probabilities
  // the CTA's first chunk
  int32_t job, chunk;
  int32_t scan[kThreads / 32];
};

constexpr size_t smem_bytes() { return 1024 + kQBytes + 2 * kXBytes + 2 * kPBytes + sizeof(Smem); }

// A job that spans CTAs, written by the second of them: its chunks are
// [start, end) of all chunks (job -1: the CTA is no job's second one).
struct __align__(16) Split {
  int32_t job, start, end, total;
};

// Where the partial results and the split jobs lie in the workspace.
struct Scratch {
  uint32_t *status;
  Split *split;  // [G]
  float4 *ml;    // [2 * G][kH]: maximum, sum, sum of the rounded probabilities
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
  if (a.blocks) return (a.n_sel ? min(max(__ldg(a.n_sel + bt), 0), a.n_blocks) : a.n_blocks) << shift;
  bool cut;
  return max(cut_len(__ldg(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T), 0);
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

// Whether the phase with `parity` has completed, without waiting.
__device__ __forceinline__ bool test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0u;
}
__device__ __forceinline__ bool ready(uint64_t *bar, uint32_t parity) {  // the same answer in all lanes
  return __all_sync(0xFFFFFFFFu, test(bar, parity));
}

// tc::mbar_wait with its loop kept rolled.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile uint32_t *abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < tc::kWaitLimit; i++) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
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

// S of 16 heads x 64 rows: lane l holds heads l/4 (regs 4u, 4u+1) and l/4 + 8
// (regs 4u+2, 4u+3), rows 8u + 2 (l % 4) and the next.
__device__ __forceinline__ void tmem_ld_s(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
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

// Stored bytes of one 64-dim slab: 16-byte pieces a row, and the dims a piece holds.
template <int kFmt>
struct Fmt {
  static constexpr int kPieces = kFmt == LIDX_E2M1 ? 2 : kFmt == LIDX_E4M3 ? 4 : 8;
  static constexpr int kIters = kRows * kPieces / 32;       // pieces a lane loads
  static constexpr int kRowsPerIter = 32 / kPieces;
};

// One 64-dim slab of a chunk (or kIters * kRowsPerIter rows of it, from row
// `from` on) in registers: piece it of a lane is piece lane % kPieces of row
// from + it * kRowsPerIter + lane / kPieces.
template <int kFmt, int kIters = Fmt<kFmt>::kIters>
struct Slab {
  uint4 v[kIters];
  uint32_t scale[kFmt == LIDX_BF16 ? 1 : kIters];

  // rows: the chunk's pool rows in shared memory
  __device__ __forceinline__ void load(const void *plane, int64_t ld, const uint8_t *scales, int64_t ld_scale, int slab,
                                       int lane, const int32_t *rows, int from) {
    using F = Fmt<kFmt>;
    const uint8_t *base = static_cast<const uint8_t *>(plane) + slab * (F::kPieces * 16) + (lane % F::kPieces) * 16;
    const int64_t pitch = kFmt == LIDX_BF16 ? 2 * ld : ld;
#pragma unroll
    for (int it = 0; it < kIters; it++) {
      const int32_t p = rows[from + it * F::kRowsPerIter + lane / F::kPieces];
      v[it] = make_uint4(0, 0, 0, 0);
      if (kFmt != LIDX_BF16) scale[it] = 127u;
      if (p >= 0) {
        v[it] = __ldg(reinterpret_cast<const uint4 *>(base + p * pitch));
        if (kFmt == LIDX_E2M1) scale[it] = __ldg(scales + p * ld_scale + slab * 2 + lane % 2);
        if (kFmt == LIDX_E4M3) scale[it] = __ldg(scales + p * ld_scale + slab);
      }
    }
  }

  // expanded to bf16 into the slab's panel of X
  __device__ __forceinline__ void store(uint8_t *panel, int lane, int from) const {
    using F = Fmt<kFmt>;
#pragma unroll
    for (int it = 0; it < kIters; it++) {
      const int r = from + it * F::kRowsPerIter + lane / F::kPieces, piece = lane % F::kPieces;
      uint8_t *row = panel + r * 128;
      const uint32_t w[4] = {v[it].x, v[it].y, v[it].z, v[it].w};
      if (kFmt == LIDX_BF16) {
        *reinterpret_cast<uint4 *>(row + ((piece ^ (r & 7)) << 4)) = v[it];
      } else if (kFmt == LIDX_E2M1) {
        const E2m1Scale s(scale[it]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          uint32_t o[4];
          s.expand(w[i], o);
          *reinterpret_cast<uint4 *>(row + (((4 * piece + i) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
        const uint32_t s = e8m0_to_bf16x2(scale[it]);
#pragma unroll
        for (int i = 0; i < 2; i++)
          *reinterpret_cast<uint4 *>(row + (((2 * piece + i) ^ (r & 7)) << 4)) =
              make_uint4(mul_bf16x2(e4m3x2_to_bf16x2(w[2 * i]), s), mul_bf16x2(e4m3x2_to_bf16x2(w[2 * i] >> 16), s),
                         mul_bf16x2(e4m3x2_to_bf16x2(w[2 * i + 1]), s),
                         mul_bf16x2(e4m3x2_to_bf16x2(w[2 * i + 1] >> 16), s));
      }
    }
  }
};

// Pool row of entry e of a job's row list, or -1.
__device__ __forceinline__ int32_t entry_row(const lidx_paged_attn_args &a, int32_t bt, int shift, int32_t e,
                                             int32_t seen, int32_t n_list, bool &bounds) {
  if (e >= n_list) return -1;
  int32_t r = e, b = bt / a.T;
  if (a.blocks) {
    const int32_t j = __ldg(a.blocks + static_cast<int64_t>(bt) * a.ld_blocks + (e >> shift));
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
      tc::mbar_init(&sm->ring_free[i], kSoftmaxWarps + kLoaders + 1);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      tc::mbar_init(&sm->x_full[i], kLoaders);
      tc::mbar_init(&sm->x_free[i], 1);
      tc::mbar_init(&sm->p_full[i], kSoftmaxWarps);
    }
    tc::mbar_init(&sm->s_full, 1);
    tc::mbar_init(&sm->s_free, kSoftmaxWarps);
    tc::mbar_init(&sm->o_free, kSoftmaxWarps);
    tc::mbar_init(&sm->drained, 1);
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
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) {  // lane 0 waits; its view becomes the warp's
    bool in = true;
    if (lane == 0) in = wait_for(bar, parity, abort_flag);
    in = __shfl_sync(0xFFFFFFFFu, in, 0);
    __syncwarp();
    return in;
  };

  if (warp == kScout) {
    // -------------------------------------------------------------- scout
    int32_t job = 0, c = 0, left = 0, seen = 0, rows = 0;  // `left` chunks of the job from chunk c on
    bool bounds = false, whole = false;
    if (n > 0) {
      job = sm->job;
      c = sm->chunk;
    }
    if (lane == 0) {  // does a job that began in the CTA before continue here, and is this its second CTA?
      Split sp;
      sp.job = -1;
      sp.start = my0 - c;
      sp.end = 0;
      sp.total = total;
      const Deal deal(total, jobs.G);
      if (c > 0 && deal.start(static_cast<int32_t>(blockIdx.x) - 1) <= sp.start) {
        sp.job = job;
        sp.end = sp.start + (job_rows(a, job, gs, shift) + kRows - 1) / kRows;
      }
      ws.split[blockIdx.x] = sp;
    }
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
        seen = cut_len(__ldg(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T);
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
    if (bounds) raise_status(ws.status, LIDX_DEV_BOUNDS);
  } else if (warp >= kSoftmaxWarps && warp < kMma) {
    // ------------------------------------------------------------ loaders
    const int slab = warp - kSoftmaxWarps;
    const lidx_kv &kv = a.cache.rows;
    constexpr bool kQuant = kFmt != LIDX_BF16;
    Slab<kFmt> part;
    Slab<LIDX_BF16, 2> rope;  // the quantised formats' RoPE dims: eight rows a warp
#pragma unroll 1
    for (int i = 0; i <= n; i++) {  // chunk i - 1 into shared memory, chunk i into registers
      if (i > 0) {
        const int stage = (i - 1) & 1;
        if (i > 2 && !warp_wait(&sm->x_free[stage], (((i - 1) >> 1) - 1) & 1)) break;
        uint8_t *x = sX + stage * kXBytes;
        if (!kQuant || slab < 7) part.store(x + slab * kPanel, lane, 0);
        if (kQuant) rope.store(x + 7 * kPanel, lane, 8 * slab);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->x_full[stage]);
      }
      if (i < n) {
        const int slot = i % kRing;
        if (!warp_wait(&sm->ring_full[slot], (i / kRing) & 1)) break;
        const int32_t *rows = sm->ring[slot].row;
        if (!kQuant || slab < 7) part.load(kv.data, kv.ld, kv.scale, kv.ld_scale, slab, lane, rows, 0);
        if (kQuant) rope.load(kv.rope, kv.ld_rope, nullptr, 0, 0, lane, rows, 8 * slab);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->ring_free[slot]);
      }
    }
  } else if (warp == kMma) {
    // ------------------------------------------------- the matrix products
    // The whole warp goes through the loop, so that descriptors and flags stay
    // in uniform registers, and one elected lane issues: with a single lane in
    // the loop each product took 100 cycles to issue, whatever its shape.
    const uint32_t idesc_s = tc::idesc_bf16(64, 64), idesc_o = tc::idesc_bf16(128, 64, true, false);
    const uint64_t q_desc = tc::desc_kmajor_sw128(tc::smem_u32(sQ));
    const uint64_t x_desc = tc::desc_kmajor_sw128(tc::smem_u32(sX));
    const uint64_t xt_desc = tc::desc_mnmajor_sw128(tc::smem_u32(sX), kPanel, 1024);
    const uint64_t p_desc = tc::desc_kmajor_sw128(tc::smem_u32(sP));
    int si = 0, oi = 0;                  // the next chunk of S and of O
    int s_jobs = 0, o_jobs = 0;          // jobs begun by then
    uint32_t firsts = 0u;                // bit i % 2: chunk i is the first of its job
    int state = 0;                       // of chunk si: 0 unknown, 1 known and Q wanted, 2 Q on its way, 3 Q there
    uint32_t idle = 0;
#pragma unroll 1
    while (oi < n) {
      bool moved = false;
      if (si < n && si < oi + 2) {
        if (state == 0 && ready(&sm->ring_full[si % kRing], (si / kRing) & 1)) {
          const Chunk &k = sm->ring[si % kRing];
          state = (k.flags & kFirst) ? 1 : 3;
          firsts = (firsts & ~(1u << (si & 1))) | ((k.flags & kFirst) << (si & 1));
          if (state == 3) {
            __syncwarp();
            if (elect()) tc::mbar_arrive(&sm->ring_free[si % kRing]);
          }
        }
        if (state == 1 && (si == 0 || ready(&sm->s_full, (si - 1) & 1))) {  // Q has been read for the last time
          const int32_t job = sm->ring[si % kRing].job;
          __syncwarp();
          if (elect()) {
            tc::mbar_arrive(&sm->ring_free[si % kRing]);
            tc::mbar_arrive_expect_tx(&sm->q_full, kQBytes);
#pragma unroll 1
            for (int p = 0; p < 8; p++)
              tma_load_3d(sQ + p * kPanel, &tm_q, &sm->q_full, 64 * p, (job & ((1 << gs) - 1)) * kH, job >> gs);
          }
          __syncwarp();
          s_jobs++;
          state = 2;
        }
        if (state == 2 && ready(&sm->q_full, (s_jobs - 1) & 1)) state = 3;
        if (state == 3 && ready(&sm->x_full[si & 1], (si >> 1) & 1) && (si == 0 || ready(&sm->s_free, (si - 1) & 1))) {
          tc::tc_fence_after();
          // step k: panel k / 4, 32 bytes (k % 4) into it; part p sums panels 2p and 2p + 1
          const uint64_t xd = x_desc + (si & 1) * (kXBytes >> 4);
          if (elect()) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
#pragma unroll
              for (int part = 0; part < kParts; part++) {
                const uint32_t off = (2 * part + (j >> 2)) * (kPanel >> 4) + (j & 3) * 2;
                tc::mma_bf16(tmem + 64 * part, q_desc + off, xd + off, idesc_s, j > 0);
              }
            }
            tc::mma_commit(&sm->s_full);
          }
          __syncwarp();
          si++;
          state = 0;
          moved = true;
        }
      }
      if (oi < si && ready(&sm->p_full[oi & 1], (oi >> 1) & 1)) {
        const bool first = (firsts >> (oi & 1)) & 1u;
        if (!first || o_jobs == 0 || ready(&sm->o_free, (o_jobs - 1) & 1)) {
          tc::tc_fence_after();
          const uint64_t xd = xt_desc + (oi & 1) * (kXBytes >> 4), pd = p_desc + (oi & 1) * (kPBytes >> 4);
          if (elect()) {
#pragma unroll
            for (int kk = 0; kk < kRows / 16; kk++) {
#pragma unroll
              for (int dt = 0; dt < 4; dt++)
                tc::mma_bf16(tmem + kOCol + 64 * dt, xd + ((2 * dt * kPanel + kk * 2048) >> 4), pd + kk * 2, idesc_o,
                             !first || kk > 0);
            }
            tc::mma_commit(&sm->x_free[oi & 1]);
          }
          __syncwarp();
          o_jobs += first;
          oi++;
          moved = true;
        }
      }
      idle = moved ? 0u : idle + 1u;
      if (idle > kIdleLimit) *abort_flag = 1u;
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0u)) break;
    }
    if (oi < n) {  // a wait gave up: the copies and products in flight end before the CTA does
      volatile uint32_t unused = 0;
      if (state >= 2 && s_jobs > 0) wait_for(&sm->q_full, (s_jobs - 1) & 1, &unused);
      if (elect()) tc::mma_commit(&sm->drained);
      __syncwarp();
      wait_for(&sm->drained, 0, &unused);
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
      cut_len(__ldg(a.len + bt / a.T), a.cache, cut);
      if (cut && tid == 0) raise_status(ws.status, LIDX_DEV_BOUNDS);
    }
    const int h0 = warp * 16 + (lane >> 2), h1 = h0 + 8;  // this lane's heads
    // logits are s * c2 in base 2; with a negative scale s changes sign instead, and a zero one
    // becomes one that makes every product round away (0 * -inf would be NaN)
    const bool negative = a.scale < 0.f;
    const float c2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
    const uint32_t quarter = static_cast<uint32_t>(warp * 32) << 16;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, r0 = 0.f, r1 = 0.f;  // r: of the rounded probabilities
    bool first_segment = true;  // the CTA's first job
    // After a wait that gave up the warp goes through the rest of its chunks
    // without touching TMEM or global memory, for the others' barriers.
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < n; i++) {
      const int stage = i & 1, slot = i % kRing;
      ok = warp_wait(&sm->ring_full[slot], (i / kRing) & 1) && ok;
      const uint32_t v0 = sm->ring[slot].valid[0], v1 = sm->ring[slot].valid[1];
      const int32_t job = sm->ring[slot].job;
      const uint32_t flags = ok ? sm->ring[slot].flags : 0u;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->ring_free[slot]);
      ok = warp_wait(&sm->s_full, i & 1) && ok;
      float s0[16], s1[16];
      if (ok) {
        tc::tc_fence_after();
        uint32_t x[32], y[32];
#pragma unroll
        for (int part = 0; part < kParts; part += 2) {
          tmem_ld_s(tmem + quarter + 64 * part, x);
          tmem_ld_s(tmem + quarter + 64 * (part + 1), y);
          tc::tmem_ld_wait();
          tc::tmem_ld32_pin(x);
          tc::tmem_ld32_pin(y);
#pragma unroll
          for (int u = 0; u < 16; u++) {
            const int k = 4 * (u >> 1) + (u & 1);
            const float p = __uint_as_float(x[k]) + __uint_as_float(y[k]);
            const float q = __uint_as_float(x[k + 2]) + __uint_as_float(y[k + 2]);
            s0[u] = part ? s0[u] + p : p;
            s1[u] = part ? s1[u] + q : q;
          }
        }
        tc::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->s_free);
      float t0 = -INFINITY, t1 = -INFINITY;
      if (negative || (v0 & v1) != 0xFFFFFFFFu) {
#pragma unroll
        for (int u = 0; u < 16; u++) {  // row 8 (u / 2) + 2 (lane % 4) + u % 2
          const uint32_t bits = (u < 8 ? v0 : v1) >> (2 * (lane & 3));
          const bool in = (bits >> (8 * ((u >> 1) & 3) + (u & 1))) & 1u;
          s0[u] = in ? (negative ? -s0[u] : s0[u]) : -INFINITY;
          s1[u] = in ? (negative ? -s1[u] : s1[u]) : -INFINITY;
        }
      }
#pragma unroll
      for (int u = 0; u < 16; u++) {
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
      // the reference maximum moves only on rises above kLazy (the first rise
      // from -inf finds an O of zeros: nothing to rescale)
      const float n0 = t0 <= m0 + kLazy ? m0 : fmaxf(t0, m0), n1 = t1 <= m1 + kLazy ? m1 : fmaxf(t1, m1);
      const float a0 = n0 == m0 || m0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
      const float a1 = n1 == m1 || m1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= a0;
      l1 *= a1;
      r0 *= a0;
      r1 *= a1;
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      if ((lane & 3) == 0) {
        sm->alpha[stage][h0] = a0;
        sm->alpha[stage][h1] = a1;
      }
      const uint32_t moved = bar_or(1, 32 * kSoftmaxWarps, a0 != 1.f || a1 != 1.f);
      if (moved) ok = warp_wait(&sm->x_free[stage ^ 1], ((i - 1) >> 1) & 1) && ok;
      if (moved && ok) {  // rescale O^T: lane = dim, columns = heads; the last second product is done
        tc::tc_fence_after();
#pragma unroll 1
        for (int q = 0; q < 16; q++) {
          const uint32_t ta = tmem + quarter + kOCol + 16 * q;
          float v[16];
          tc::tmem_ld16(ta, v);
#pragma unroll
          for (int h = 0; h < 16; h++) v[h] *= sm->alpha[stage][16 * (q & 3) + h];
          tmem_st16(ta, v);
        }
        tmem_st_wait();
      }
      // P^T line `head`: 16-byte pieces of eight rows, swizzled with head & 7 (free once chunk i - 2 is done)
      if (i >= 2) ok = warp_wait(&sm->x_free[stage], ((i >> 1) - 1) & 1) && ok;
      uint8_t *p0 = sP + stage * kPBytes + h0 * 128 + 4 * (lane & 3), *p1 = p0 + 8 * 128;
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const float x0 = exp2_approx(fmaf(s0[2 * u], c2, -b0)), x1 = exp2_approx(fmaf(s0[2 * u + 1], c2, -b0));
        const float y0 = exp2_approx(fmaf(s1[2 * u], c2, -b1)), y1 = exp2_approx(fmaf(s1[2 * u + 1], c2, -b1));
        l0 += x0 + x1;
        l1 += y0 + y1;
        const __nv_bfloat162 px = __floats2bfloat162_rn(x0, x1), py = __floats2bfloat162_rn(y0, y1);
        const uint32_t wx = *reinterpret_cast<const uint32_t *>(&px), wy = *reinterpret_cast<const uint32_t *>(&py);
        r0 += bf16x2_lo(wx) + bf16x2_hi(wx);
        r1 += bf16x2_lo(wy) + bf16x2_hi(wy);
        *reinterpret_cast<uint32_t *>(p0 + ((u ^ (h0 & 7)) << 4)) = wx;
        *reinterpret_cast<uint32_t *>(p1 + ((u ^ (h0 & 7)) << 4)) = wy;
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->p_full[stage]);

      if (flags & kLast) {  // this CTA's part of the job is done
        const int32_t bt = job >> gs, g = job & ((1 << gs) - 1);
        const bool out_now = flags & kWhole;
        ok = warp_wait(&sm->x_free[stage], (i >> 1) & 1) && ok;
        tc::tc_fence_after();
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
          l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
          r0 += __shfl_xor_sync(0xFFFFFFFFu, r0, o);
          r1 += __shfl_xor_sync(0xFFFFFFFFu, r1, o);
        }
        const int heads = min(kH, a.H - g * kH);
        const int64_t out_row = static_cast<int64_t>(bt) * a.H + g * kH;
        const int64_t slot_o = 2 * static_cast<int64_t>(blockIdx.x) + (first_segment ? 0 : 1);
        if ((lane & 3) < 2 && ok) {
          const int h = (lane & 1) ? h1 : h0;
          const float m = (lane & 1) ? m1 : m0, l = (lane & 1) ? l1 : l0, rounded = (lane & 1) ? r1 : r0;
          if (out_now) {
            sm->l[h] = rounded == 0.f ? 0.f : 1.f / rounded;
            if (a.lse && h < heads) a.lse[out_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            ws.ml[slot_o * kH + h] = make_float4(m, l, rounded, 0.f);
          }
        }
        bar_or(1, 32 * kSoftmaxWarps, 0u);  // sm->l is in
#pragma unroll 1
        for (int q = 0; q < 16 && ok; q++) {  // 16 heads of a dim tile at a time
          const int d = 128 * (q >> 2) + 32 * warp + lane, hb = 16 * (q & 3);
          float v[16];
          tc::tmem_ld16(tmem + quarter + kOCol + 16 * q, v);
          if (out_now) {
            // an 8 x 8 exchange among eight lanes: lane = dim, registers = heads, to a lane with eight dims of a head
            uint32_t w1[8], w2[8], w3[8];
            const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;  // odd: other's high, own high half; even: own low, other's low
#pragma unroll
            for (int k = 0; k < 8; k++) {
              const __nv_bfloat162 two =
                  __floats2bfloat162_rn(v[2 * k] * sm->l[hb + 2 * k], v[2 * k + 1] * sm->l[hb + 2 * k + 1]);
              const uint32_t own = *reinterpret_cast<const uint32_t *>(&two);
              w1[k] = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), pick);  // head 2k + lane % 2
            }
#pragma unroll
            for (int k = 0; k < 4; k++) {  // head 4k + lane % 4: words 2k, 2k + 1
              const bool odd = lane & 2;
              const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? w1[2 * k] : w1[2 * k + 1], 2);
              w2[2 * k] = odd ? other : w1[2 * k];
              w2[2 * k + 1] = odd ? w1[2 * k + 1] : other;
            }
            uint16_t *o = static_cast<uint16_t *>(a.out) + (out_row + hb + (lane & 7)) * kD + (d & ~7);
#pragma unroll
            for (int k = 0; k < 2; k++) {  // head 8k + lane % 8: words 4k .. 4k + 3
              const bool odd = lane & 4;
#pragma unroll
              for (int j = 0; j < 2; j++) {
                const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? w2[4 * k + j] : w2[4 * k + 2 + j], 4);
                w3[4 * k + j] = odd ? other : w2[4 * k + j];
                w3[4 * k + 2 + j] = odd ? w2[4 * k + 2 + j] : other;
              }
              if (hb + 8 * k + (lane & 7) < heads)
                *reinterpret_cast<uint4 *>(o + 8 * k * kD) = make_uint4(w3[4 * k], w3[4 * k + 1], w3[4 * k + 2], w3[4 * k + 3]);
            }
          } else {
            float4 *o = ws.o + (slot_o * (kH / 4) + hb / 4) * kD + d;
#pragma unroll
            for (int k = 0; k < 4; k++) o[k * kD] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->o_free);
        m0 = m1 = -INFINITY;
        l0 = l1 = r0 = r1 = 0.f;
        first_segment = false;
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
// weights are found, a thread for each partial, then the weighted sum runs
// over the partials.  Where a job has few of them, as with many short jobs, a
// warp joins an item by itself; where it has many, the eight warps of the CTA
// take every eighth partial each and their sums meet in shared memory.
__global__ void __launch_bounds__(kMergeThreads) paged_attn_merge_kernel(const lidx_paged_attn_args a, const Jobs jobs,
                                                                         const Scratch ws) {
  constexpr int kWarps = kMergeThreads / 32, kItems = (kH / 4) * (kD / 32);
  __shared__ Split list[kMaxCtas];  // jobs with few partials from the front, with many from the back
  __shared__ int32_t count[2][kWarps];
  __shared__ float4 weight_s[kMaxCtas], acc_s[kWarps][32], red_s[3][kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();  // the partial results come from the previous kernel
  // the split jobs, in the same order in every CTA (kMaxCtas <= kMergeThreads)
  Split sp;
  sp.job = -1;
  if (tid < jobs.G) sp = ws.split[tid];
  bool many = false;
  if (sp.job >= 0) {
    const Deal deal(sp.total, jobs.G);
    many = deal.owner(sp.end - 1) - deal.owner(sp.start) >= kFew;
  }
  const uint32_t few_mask = __ballot_sync(0xFFFFFFFFu, sp.job >= 0 && !many), many_mask = __ballot_sync(0xFFFFFFFFu, many);
  if (lane == 0) {
    count[0][warp] = __popc(few_mask);
    count[1][warp] = __popc(many_mask);
  }
  __syncthreads();
  int n_few = 0, n_many = 0, at = __popc((many ? many_mask : few_mask) & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) at += count[many][w];
    n_few += count[0][w];
    n_many += count[1][w];
  }
  if (sp.job >= 0) list[many ? kMaxCtas - 1 - at : at] = sp;
  __syncthreads();

  float m[4], l[4], r[4], e[4];  // of four heads of the partial that the thread looks after
  auto look = [&](const float4 *ml) {
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float4 x = ml ? ml[k] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      m[k] = x.x;
      l[k] = x.y;
      r[k] = x.z;
    }
  };
  // the job is the CTA's first one unless the CTA began with an earlier job
  auto slot_of = [&](const Deal &deal, int32_t c, int32_t start) { return 2 * c + (deal.start(c) < start ? 1 : 0); };
  auto write = [&](const Split &sj, int h, int d0, float M, float L, float R, float A) {  // head h of the job's group
    const int32_t bt = sj.job >> jobs.group_shift, group = sj.job & ((1 << jobs.group_shift) - 1);
    if (group * kH + h >= a.H) return;
    const int64_t row = static_cast<int64_t>(bt) * a.H + group * kH + h;
    static_cast<__nv_bfloat16 *>(a.out)[row * kD + d0 + lane] = __float2bfloat16_rn(A * (R == 0.f ? 0.f : 1.f / R));
    if (a.lse && d0 == 0 && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  };

#pragma unroll 1
  for (int item = blockIdx.x * kWarps + warp; item < n_few * kItems / 4; item += gridDim.x * kWarps) {  // 128 dims each
    const Split sj = list[item / (kItems / 4)];
    const int h4 = (item % (kItems / 4)) / 4, d0 = 128 * (item % 4);
    const Deal deal(sj.total, jobs.G);
    const int32_t from = deal.owner(sj.start), last = deal.owner(sj.end - 1);
    float M[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, L[4] = {0.f, 0.f, 0.f, 0.f}, R[4] = {0.f, 0.f, 0.f, 0.f}, A[4][4] = {};
#pragma unroll 1
    for (int32_t c = from; c <= last; c++) {
      look(ws.ml + slot_of(deal, c, sj.start) * kH + 4 * h4);
#pragma unroll
      for (int k = 0; k < 4; k++) M[k] = fmaxf(M[k], m[k]);
    }
#pragma unroll 2
    for (int32_t c = from; c <= last; c++) {
      const int32_t slot = slot_of(deal, c, sj.start);
      look(ws.ml + slot * kH + 4 * h4);
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; j++) v[j] = ws.o[static_cast<size_t>(slot * (kH / 4) + h4) * kD + d0 + 32 * j + lane];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float e0 = weight_of(m[k], M[k]);
        L[k] = fmaf(e0, l[k], L[k]);
        R[k] = fmaf(e0, r[k], R[k]);
#pragma unroll
        for (int j = 0; j < 4; j++) A[k][j] = fmaf(e0, reinterpret_cast<const float *>(&v[j])[k], A[k][j]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
#pragma unroll
      for (int j = 0; j < 4; j++) write(sj, 4 * h4 + k, d0 + 32 * j, M[k], L[k], R[k], A[k][j]);
  }

#pragma unroll 1
  for (int item = blockIdx.x; item < n_many * kItems; item += gridDim.x) {
    const Split sj = list[kMaxCtas - 1 - item / kItems];
    const int h4 = (item % kItems) / (kD / 32), d0 = 32 * (item % (kD / 32));
    const Deal deal(sj.total, jobs.G);
    const int32_t from = deal.owner(sj.start), n = deal.owner(sj.end - 1) - from + 1;  // <= kMaxCtas
    look(tid < n ? ws.ml + slot_of(deal, from + tid, sj.start) * kH + 4 * h4 : nullptr);
    float M[4], L[4], R[4];
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
      R[k] = warp_sum(tid < n ? e[k] * r[k] : 0.f);
    }
    if (tid < n) weight_s[tid] = make_float4(e[0], e[1], e[2], e[3]);
    if (lane == 0) {
      red_s[1][warp] = make_float4(L[0], L[1], L[2], L[3]);
      red_s[2][warp] = make_float4(R[0], R[1], R[2], R[3]);
    }
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int32_t c = warp; c < n; c += kWarps) {
      const float4 v = ws.o[static_cast<size_t>(slot_of(deal, from + c, sj.start) * (kH / 4) + h4) * kD + d0 + lane];
      const float4 w = weight_s[c];
      acc.x = fmaf(w.x, v.x, acc.x);
      acc.y = fmaf(w.y, v.y, acc.y);
      acc.z = fmaf(w.z, v.z, acc.z);
      acc.w = fmaf(w.w, v.w, acc.w);
    }
    acc_s[warp][lane] = acc;
    __syncthreads();
    if (warp < 4) {  // warp k finishes head k
      float A = 0.f, Ls = 0.f, Rs = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        A += reinterpret_cast<const float *>(&acc_s[w][lane])[warp];
        Ls += reinterpret_cast<const float *>(&red_s[1][w])[warp];
        Rs += reinterpret_cast<const float *>(&red_s[2][w])[warp];
      }
      write(sj, 4 * h4 + warp, d0, warp == 0 ? M[0] : warp == 1 ? M[1] : warp == 2 ? M[2] : M[3], Ls, Rs, A);
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
  return rows <= INT32_MAX && job_count(a) <= (1 << 24) && job_count(a) * most_chunks(a) <= INT32_MAX;
}

size_t paged_attn_workspace(const lidx_paged_attn_args &a) {
  const Jobs j = plan(a);
  return LIDX_WS_HEADER + align256(j.G * sizeof(Split)) + static_cast<size_t>(j.G) * 2 * kH * (sizeof(float4) + kD * 4);
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
  s.ml = reinterpret_cast<float4 *>(p);
  p += static_cast<size_t>(j.G) * 2 * kH * sizeof(float4);
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
  return launch_kernel(paged_attn_merge_kernel, dim3(4 * sm_count()), dim3(kMergeThreads), 0, st, true, a, j, s);
}

}  // namespace lidx
