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
// A chunk, in a CTA of 13 warps:
//   * eight loader warps, one per 64-dim slab of the row, fetch the stored
//     rows one to two chunks ahead into registers, expand them to bf16 (exact:
//     every E2M1 or E4M3 value times a power of two is a bf16 value) and store
//     them as the swizzled K-major tile X[64 rows][512], two of which are in
//     shared memory.  Rows that are not attended to are stored as zeros.
//   * one thread issues S[head][row] = Q . X^T (M = 64, N = 64, K = 512) and,
//     when the chunk's probabilities are there, O^T[d][head] += X^T . P^T
//     (M = 128 four times, N = 64, K = 64), both on tcgen05 with fp32
//     accumulators in TMEM; S is double buffered, so the S of a chunk runs
//     while the softmax of the one before it does.
//   * four softmax warps read S in the 16x256b shape, in which the 32 lanes of
//     a warp share the 16 heads of its TMEM quarter (8 head pairs x 4 column
//     groups), so row maxima take two shuffles and no lane idles.  The running
//     maximum moves only when it rises by more than 8 (base 2); then the O so
//     far is rescaled in TMEM.  Sums are of the fp32 probabilities.
//   P is rounded to bf16 for the second product: 2^-9 of each probability,
//   independent errors that average out to less than the bf16 output's own
//   rounding.
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
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoaders + 1);
constexpr int kPanel = 64 * 128;         // one 64-line panel of X or Q: 64 dims
constexpr int kXBytes = 8 * kPanel;
constexpr int kQBytes = 8 * kPanel;
constexpr int kPBytes = kH * kRows * 2;
constexpr uint32_t kSCol = 0;            // S buffer i at columns 64 i
constexpr uint32_t kOCol = 128;          // O^T tile t at columns kOCol + 64 t
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.f;             // base-2 headroom of the reference maximum
constexpr int kMergeThreads = 256;
constexpr int kMaxCtas = 256;            // one CTA per SM

struct __align__(8) Smem {
  uint64_t q_full;
  uint64_t x_full[2], x_free[2];  // a stage's rows are in / its second product is done (X and P free again)
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2];
  uint64_t o_free;                // the finished job's O has been read
  uint64_t drained;               // every product issued is done (only after a wait gave up)
  uint64_t valid[2];              // bit r: row r of the stage's chunk is attended to
  uint32_t tmem_base;
  uint32_t abort;
  float alpha[2][kH];             // rescale factors of a chunk
  float m[kH], l[kH];
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
  float2 *ml;    // [2 * G][kH]
  float *o;      // [2 * G][kH][kD]
};

// The job list.
struct Jobs {
  int32_t n;       // B * T * groups of heads
  int32_t groups;  // of 64 heads
  int32_t G;       // CTAs
};

__device__ __forceinline__ int32_t range_start(int32_t g, int32_t G, int32_t total) {
  return static_cast<int32_t>(static_cast<int64_t>(g) * total / G);
}

// the CTA that holds chunk c
__device__ __forceinline__ int32_t owner(int32_t c, int32_t G, int32_t total) {
  return static_cast<int32_t>(((static_cast<int64_t>(c) + 1) * G - 1) / total);
}

// Entries of job's row list: rows for the dense case, rows of the listed blocks otherwise.
__device__ __forceinline__ int32_t job_rows(const lidx_paged_attn_args &a, int32_t job, int groups, int shift) {
  const int32_t bt = job / groups;
  if (a.blocks) return (a.n_sel ? min(max(__ldg(a.n_sel + bt), 0), a.n_blocks) : a.n_blocks) << shift;
  bool cut;
  return max(cut_len(__ldg(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T), 0);
}
__device__ __forceinline__ int32_t job_chunks(const lidx_paged_attn_args &a, int32_t job, int groups, int shift) {
  return (job_rows(a, job, groups, shift) + kRows - 1) / kRows;
}

// Walks the CTA's chunks: `left` of them from chunk c of job on.
struct Cursor {
  int32_t job, c, n, left;  // n: chunks of the job
  __device__ __forceinline__ void next(const lidx_paged_attn_args &a, int groups, int shift) {
    left--;
    if (++c < n) return;
    c = 0;
    while (left > 0) {
      n = job_chunks(a, ++job, groups, shift);
      if (n > 0) return;
    }
  }
};

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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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

// One 64-dim slab of a chunk in registers: piece it of a lane is piece
// lane % kPieces of row it * kRowsPerIter + lane / kPieces.
template <int kFmt, int kIters = Fmt<kFmt>::kIters>
struct Slab {
  uint4 v[kIters];
  uint32_t scale[kFmt == LIDX_BF16 ? 1 : kIters];

  // pool rows of rows lane and lane + 32 of the chunk are p0 and p1 (-1: none);
  // `from`: first row, for a part of a chunk (kIters < Fmt::kIters)
  __device__ __forceinline__ void load(const void *plane, int64_t ld, const uint8_t *scales, int64_t ld_scale, int slab,
                                       int lane, int32_t p0, int32_t p1, int from) {
    using F = Fmt<kFmt>;
    const uint8_t *base = static_cast<const uint8_t *>(plane) + slab * (F::kPieces * 16) + (lane % F::kPieces) * 16;
    const int64_t pitch = kFmt == LIDX_BF16 ? 2 * ld : ld;
#pragma unroll
    for (int it = 0; it < kIters; it++) {
      const int r = from + it * F::kRowsPerIter + lane / F::kPieces;
      const int32_t a0 = __shfl_sync(0xFFFFFFFFu, p0, r & 31), a1 = __shfl_sync(0xFFFFFFFFu, p1, r & 31);
      const int32_t p = r < 32 ? a0 : a1;
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
        const uint32_t s = e8m0_to_bf16x2(scale[it]);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          uint32_t o[4];
          e2m1x8_to_bf16x2(w[i], o);
          *reinterpret_cast<uint4 *>(row + (((4 * piece + i) ^ (r & 7)) << 4)) =
              make_uint4(mul_bf16x2(o[0], s), mul_bf16x2(o[1], s), mul_bf16x2(o[2], s), mul_bf16x2(o[3], s));
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = jobs.groups;

  if (tid == 0) {
    tc::mbar_init(&sm->q_full, 1);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      tc::mbar_init(&sm->x_full[i], kLoaders);
      tc::mbar_init(&sm->x_free[i], 1);
      tc::mbar_init(&sm->s_full[i], 1);
      tc::mbar_init(&sm->s_free[i], kSoftmaxWarps);
      tc::mbar_init(&sm->p_full[i], kSoftmaxWarps);
    }
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
    for (int j = j0; j < j1; j++) mine += job_chunks(a, j, groups, shift);
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
    my0 = range_start(blockIdx.x, jobs.G, total);
    my1 = range_start(blockIdx.x + 1, jobs.G, total);
    if (before <= my0 && my0 < before + mine) {
      int32_t at = before;
      for (int j = j0; j < j1; j++) {
        const int32_t n = job_chunks(a, j, groups, shift);
        if (at <= my0 && my0 < at + n) {
          sm->job = j;
          sm->chunk = my0 - at;
        }
        at += n;
      }
    }
    __syncthreads();
  }
  Cursor cur;
  cur.left = my1 - my0;
  if (cur.left > 0) {
    cur.job = sm->job;
    cur.c = sm->chunk;
    cur.n = job_chunks(a, cur.job, groups, shift);
  }
  if (tid == 0) {
    const int32_t start = my0 - (cur.left > 0 ? cur.c : 0);
    const bool second =
        cur.left > 0 && cur.c > 0 && range_start(owner(my0 - 1, jobs.G, total), jobs.G, total) <= start;
    Split sp;
    sp.job = second ? cur.job : -1;
    sp.start = start;
    sp.end = start + (second ? cur.n : 0);
    sp.total = total;
    ws.split[blockIdx.x] = sp;
  }

  if (cur.left > 0 && warp >= kSoftmaxWarps && warp < kSoftmaxWarps + kLoaders) {
    // ------------------------------------------------------------ loaders
    const int slab = warp - kSoftmaxWarps;
    const lidx_kv &kv = a.cache.rows;
    constexpr bool kQuant = kFmt != LIDX_BF16;
    constexpr int kSets = kQuant ? 2 : 1;  // chunks in registers
    // rows of the chunk after the ones in registers
    bool bounds = false;
    int32_t last_job = -1, seen = 0, n_list = 0;
    auto find_rows = [&](const Cursor &k, int32_t &p0, int32_t &p1) {
      p0 = p1 = -1;
      if (k.left <= 0) return;
      const int32_t bt = k.job / groups;
      if (k.job != last_job) {
        last_job = k.job;
        bool cut;
        seen = cut_len(__ldg(a.len + bt / a.T), a.cache, cut) - (a.T - 1 - bt % a.T);
        bounds |= cut;
        n_list = job_rows(a, k.job, groups, shift);
      }
      p0 = entry_row(a, bt, shift, k.c * kRows + lane, seen, n_list, bounds);
      p1 = entry_row(a, bt, shift, k.c * kRows + 32 + lane, seen, n_list, bounds);
    };
    Slab<kFmt> body[kSets];
    Slab<LIDX_BF16, 2> rope[kSets];  // the quantised formats' RoPE dims: eight rows a warp
    uint64_t mask[kSets];
    auto load = [&](int set, int32_t p0, int32_t p1) {
      if (!kQuant || slab < 7) body[set].load(kv.data, kv.ld, kv.scale, kv.ld_scale, slab, lane, p0, p1, 0);
      if (kQuant) rope[set].load(kv.rope, kv.ld_rope, nullptr, 0, 0, lane, p0, p1, 8 * slab);
      mask[set] = static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, p0 >= 0)) |
                  (static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, p1 >= 0)) << 32);
    };
    const int n = cur.left;
    Cursor ahead = cur;
    int32_t p0, p1;
#pragma unroll
    for (int s = 0; s < kSets; s++) {
      find_rows(ahead, p0, p1);
      load(s, p0, p1);
      if (ahead.left > 0) ahead.next(a, groups, shift);
    }
    find_rows(ahead, p0, p1);
    auto step = [&](int i, int set) {
      const int stage = i & 1;
      bool ok = true;
      if (i >= 2) {
        if (lane == 0) ok = tc::mbar_wait(&sm->x_free[stage], ((i >> 1) - 1) & 1, abort_flag);
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        __syncwarp();
      }
      if (!ok) return false;
      uint8_t *x = sX + stage * kXBytes;
      if (!kQuant || slab < 7) body[set].store(x + slab * kPanel, lane, 0);
      if (kQuant) rope[set].store(x + 7 * kPanel, lane, 8 * slab);
      if (slab == 0 && lane == 0) sm->valid[stage] = mask[set];
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->x_full[stage]);
      load(set, p0, p1);
      if (ahead.left > 0) ahead.next(a, groups, shift);
      find_rows(ahead, p0, p1);
      return true;
    };
    for (int i = 0; i < n; i += kSets) {
      if (!step(i, 0)) break;
      if (kSets == 2 && i + 1 < n && !step(i + 1, kSets - 1)) break;
    }
    if (bounds && slab == 0) raise_status(ws.status, LIDX_DEV_BOUNDS);
  } else if (cur.left > 0 && warp == kSoftmaxWarps + kLoaders) {
    // ------------------------------------------------- the matrix products
    if (lane == 0) {
      const uint32_t qs = tc::smem_u32(sQ);
      const uint32_t idesc_s = tc::idesc_bf16(64, 64), idesc_o = tc::idesc_bf16(128, 64, true, false);
      const int n = cur.left;
      int job_no = 0;           // jobs begun so far
      int q_loads = 0;
      bool pending = false;     // the second product of chunk i - 1 is still to be issued
      bool pending_first = false;
      bool ok = true;
      auto second = [&](int i, bool first) {  // O^T (+)= X^T . P^T of chunk i
        const int stage = i & 1;
        if (first && job_no > 1) ok = ok && tc::mbar_wait(&sm->o_free, (job_no - 2) & 1, abort_flag);
        ok = ok && tc::mbar_wait(&sm->p_full[stage], (i >> 1) & 1, abort_flag);
        if (!ok) return;
        tc::tc_fence_after();
        const uint32_t xs = tc::smem_u32(sX + stage * kXBytes), ps = tc::smem_u32(sP + stage * kPBytes);
#pragma unroll
        for (int dt = 0; dt < 4; dt++)
#pragma unroll
          for (int kk = 0; kk < kRows / 16; kk++)
            tc::mma_bf16(tmem + kOCol + 64 * dt, tc::desc_mnmajor_sw128(xs + 2 * dt * kPanel + kk * 2048, kPanel, 1024),
                         tc::desc_kmajor_sw128(ps + kk * 32), idesc_o, !first || kk > 0);
        tc::mma_commit(&sm->x_free[stage]);
      };
      for (int i = 0; i < n && ok; i++) {
        const int stage = i & 1;
        const bool first = i == 0 || cur.c == 0;
        if (first) {
          // the last job's S products have read Q
          if (i > 0) ok = ok && tc::mbar_wait(&sm->s_full[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag);
          if (ok) {
            tc::mbar_arrive_expect_tx(&sm->q_full, kQBytes);
            q_loads++;
#pragma unroll
            for (int p = 0; p < 8; p++)
              tma_load_3d(sQ + p * kPanel, &tm_q, &sm->q_full, 64 * p, (cur.job % groups) * kH, cur.job / groups);
          }
          if (pending) second(i - 1, pending_first);
          pending = false;
          ok = ok && tc::mbar_wait(&sm->q_full, job_no & 1, abort_flag);
          job_no++;
        }
        ok = ok && tc::mbar_wait(&sm->x_full[stage], (i >> 1) & 1, abort_flag);
        if (i >= 2) ok = ok && tc::mbar_wait(&sm->s_free[stage], ((i >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t xs = tc::smem_u32(sX + stage * kXBytes);
#pragma unroll
        for (int k = 0; k < kD / 16; k++) {
          const uint32_t off = (k >> 2) * kPanel + (k & 3) * 32;
          tc::mma_bf16(tmem + kSCol + 64 * stage, tc::desc_kmajor_sw128(qs + off), tc::desc_kmajor_sw128(xs + off),
                       idesc_s, k > 0);
        }
        tc::mma_commit(&sm->s_full[stage]);
        if (pending) second(i - 1, pending_first);
        pending = true;
        pending_first = first;
        cur.next(a, groups, shift);
      }
      if (pending && ok) second(n - 1, pending_first);
      // a wait that gave up may leave copies and products in flight: they end before the CTA does
      if (!ok) {
        volatile uint32_t unused = 0;
        if (q_loads > 0) tc::mbar_wait(&sm->q_full, (q_loads - 1) & 1, &unused);
        tc::mma_commit(&sm->drained);
        tc::mbar_wait(&sm->drained, 0, &unused);
      }
    }
  } else if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    // first, while the first rows are on their way: the jobs without rows, dealt out to the CTAs
    for (int32_t j = blockIdx.x; j < jobs.n; j += jobs.G) {
      if (job_rows(a, j, groups, shift) > 0) continue;
      const int32_t bt = j / groups, g = j % groups, heads = min(kH, a.H - g * kH);
      const int64_t row = static_cast<int64_t>(bt) * a.H + g * kH;
      uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row * kD);
      for (int i = tid; i < heads * kD / 8; i += 32 * kSoftmaxWarps) o[i] = make_uint4(0, 0, 0, 0);
      if (a.lse && tid < heads) a.lse[row + tid] = -INFINITY;
      bool cut;
      cut_len(__ldg(a.len + bt / a.T), a.cache, cut);
      if (cut && tid == 0) raise_status(ws.status, LIDX_DEV_BOUNDS);
    }
    const int h0 = warp * 16 + (lane >> 2), h1 = h0 + 8;  // this lane's heads
    const float c2 = a.scale * kLog2e;
    const uint32_t quarter = static_cast<uint32_t>(warp * 32) << 16;
    const int n = max(cur.left, 0);
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    bool whole = cur.c == 0;  // the CTA began the job at its first chunk
    bool first_segment = true;
    bool fresh = true;        // nothing of the job is in O yet
    // After a wait that gave up the warp goes through the rest of its chunks
    // without touching TMEM or global memory, for the others' barriers.
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      bool in = true;
      if (lane == 0) in = tc::mbar_wait(bar, parity, abort_flag);
      in = __shfl_sync(0xFFFFFFFFu, in, 0);
      __syncwarp();
      ok = ok && in;
    };
    for (int i = 0; i < n; i++) {
      const int stage = i & 1;
      const uint32_t par = (i >> 1) & 1;
      wait(&sm->x_full[stage], par);  // orders the loaders' row mask before its reads here
      const uint64_t valid = ok ? sm->valid[stage] : 0ull;
      wait(&sm->s_full[stage], par);
      uint32_t r[32];
      if (ok) {
        tc::tc_fence_after();
        tmem_ld_s(tmem + quarter + kSCol + 64 * stage, r);
        tc::tmem_ld_wait();
        tc::tmem_ld32_pin(r);
        tc::tc_fence_before();
      } else {
#pragma unroll
        for (int k = 0; k < 32; k++) r[k] = 0u;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->s_free[stage]);
      float s0[16], s1[16];
      float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const uint32_t two = static_cast<uint32_t>(valid >> (8 * u + 2 * (lane & 3)));
#pragma unroll
        for (int k = 0; k < 2; k++) {
          const bool in = (two >> k) & 1u;
          s0[2 * u + k] = in ? __uint_as_float(r[4 * u + k]) * c2 : -INFINITY;
          s1[2 * u + k] = in ? __uint_as_float(r[4 * u + 2 + k]) * c2 : -INFINITY;
          t0 = fmaxf(t0, s0[2 * u + k]);
          t1 = fmaxf(t1, s1[2 * u + k]);
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, o));
        t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, o));
      }
      // the reference maximum moves only on rises above kLazy (the first rise
      // from -inf finds an O of zeros: nothing to rescale)
      const float n0 = t0 <= m0 + kLazy ? m0 : fmaxf(t0, m0), n1 = t1 <= m1 + kLazy ? m1 : fmaxf(t1, m1);
      const float a0 = n0 == m0 || m0 == -INFINITY ? 1.f : exp2_approx(m0 - n0);
      const float a1 = n1 == m1 || m1 == -INFINITY ? 1.f : exp2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= a0;
      l1 *= a1;
      const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
      if ((lane & 3) == 0) {
        sm->alpha[stage][h0] = a0;
        sm->alpha[stage][h1] = a1;
      }
      uint32_t p0[8], p1[8];
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const float x0 = exp2_approx(s0[2 * u] - b0), x1 = exp2_approx(s0[2 * u + 1] - b0);
        const float y0 = exp2_approx(s1[2 * u] - b1), y1 = exp2_approx(s1[2 * u + 1] - b1);
        l0 += x0 + x1;
        l1 += y0 + y1;
        const __nv_bfloat162 px = __floats2bfloat162_rn(x0, x1), py = __floats2bfloat162_rn(y0, y1);
        p0[u] = *reinterpret_cast<const uint32_t *>(&px);
        p1[u] = *reinterpret_cast<const uint32_t *>(&py);
      }
      const uint32_t moved = bar_or(1, 32 * kSoftmaxWarps, !fresh && (a0 != 1.f || a1 != 1.f));
      if (moved) wait(&sm->x_free[stage ^ 1], ((i - 1) >> 1) & 1);
      if (moved && ok) {  // rescale O^T: lane = dim, columns = heads; the last second product is done
        tc::tc_fence_after();
        for (int q = 0; q < 8; q++) {
          const uint32_t ta = tmem + quarter + kOCol + 32 * q;
          uint32_t v[32];
          tc::tmem_ld32_issue(ta, v);
          tc::tmem_ld_wait();
          tc::tmem_ld32_pin(v);
#pragma unroll
          for (int h = 0; h < 32; h++)
            v[h] = __float_as_uint(__uint_as_float(v[h]) * sm->alpha[stage][32 * (q & 1) + h]);
          tmem_st32(ta, v);
        }
        tmem_st_wait();
      }
      // P^T line `head`: 16-byte pieces of eight rows, swizzled with head & 7 (free once chunk i - 2 is done)
      if (i >= 2) wait(&sm->x_free[stage], ((i >> 1) - 1) & 1);
      uint8_t *p = sP + stage * kPBytes;
#pragma unroll
      for (int u = 0; u < 8; u++) {
        *reinterpret_cast<uint32_t *>(p + h0 * 128 + ((u ^ (h0 & 7)) << 4) + 4 * (lane & 3)) = p0[u];
        *reinterpret_cast<uint32_t *>(p + h1 * 128 + ((u ^ (h1 & 7)) << 4) + 4 * (lane & 3)) = p1[u];
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm->p_full[stage]);
      fresh = false;

      const bool job_ends = cur.c + 1 == cur.n;
      if (job_ends || i + 1 == n) {
        // ---- this CTA's part of the job is done
        const int32_t bt = cur.job / groups, g = cur.job % groups;
        const bool out_now = whole && job_ends;
        wait(&sm->x_free[stage], par);
        tc::tc_fence_after();
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, o);
          l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, o);
        }
        const int heads = min(kH, a.H - g * kH);
        const int64_t out_row = static_cast<int64_t>(bt) * a.H + g * kH;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (first_segment ? 0 : 1);
        if ((lane & 3) == 0 && ok) {
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const int h = k ? h1 : h0;
            const float m = k ? m1 : m0, l = k ? l1 : l0;
            if (out_now) {
              sm->l[h] = l == 0.f ? 0.f : 1.f / l;
              if (a.lse && h < heads) a.lse[out_row + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
              ws.ml[slot * kH + h] = make_float2(m, l);
            }
          }
        }
        bar_or(1, 32 * kSoftmaxWarps, 0u);  // sm->l is in
        for (int q = 0; q < 8 && ok; q++) {
          const int d = 128 * (q >> 1) + 32 * warp + lane, hb = 32 * (q & 1);
          uint32_t v[32];
          tc::tmem_ld32_issue(tmem + quarter + kOCol + 32 * q, v);
          tc::tmem_ld_wait();
          tc::tmem_ld32_pin(v);
          if (out_now) {
            uint16_t *o = static_cast<uint16_t *>(a.out) + out_row * kD + d;
#pragma unroll
            for (int h = 0; h < 32; h++)
              if (hb + h < heads)
                o[(hb + h) * kD] = static_cast<uint16_t>(bf16_bits(__uint_as_float(v[h]) * sm->l[hb + h]));
          } else {
            float *o = ws.o + slot * kH * kD + d;
#pragma unroll
            for (int h = 0; h < 32; h++)
              if (hb + h < heads) o[(hb + h) * kD] = __uint_as_float(v[h]);
          }
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm->o_free);
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        whole = true;
        first_segment = false;
        fresh = true;
      }
      cur.next(a, groups, shift);
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

// Joins the partial results of jobs that span CTAs.  An item is such a job, a
// head and a quarter of its dims: eight warps take every eighth partial, lane
// l dims [4l, 4l + 4) of the quarter.
__global__ void __launch_bounds__(kMergeThreads) paged_attn_merge_kernel(const lidx_paged_attn_args a, const Jobs jobs,
                                                                         const Scratch ws) {
  __shared__ float4 acc_s[kMergeThreads / 32][32];
  __shared__ float2 ml_s[kMergeThreads / 32];
  __shared__ int32_t list[kMaxCtas], count[kMergeThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();  // the partial results come from the previous kernel
  // the split jobs, in the same order in every CTA (kMaxCtas <= kMergeThreads)
  const bool mine = tid < jobs.G && ws.split[tid].job >= 0;
  const uint32_t flags = __ballot_sync(0xFFFFFFFFu, mine);
  if (lane == 0) count[warp] = __popc(flags);
  __syncthreads();
  int n_list = 0, at = __popc(flags & ((1u << lane) - 1u));
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; w++) {
    if (w < warp) at += count[w];
    n_list += count[w];
  }
  if (mine) list[at] = tid;
  __syncthreads();
  constexpr int kPerJob = kH * 4;
  const int items = n_list * kPerJob;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int32_t g = list[item / kPerJob], h = (item % kPerJob) >> 2, quarter = item & 3;
    const Split sp = ws.split[g];
    const int32_t start = sp.start, end = sp.end, total = sp.total;
    const int32_t bt = sp.job / jobs.groups, group = sp.job % jobs.groups;
    if (h >= min(kH, a.H - group * kH)) continue;
    const int32_t from = owner(start, jobs.G, total), last = owner(end - 1, jobs.G, total);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int32_t c = from + warp; c <= last; c += kMergeThreads / 32) {
      const int32_t s = range_start(c, jobs.G, total);
      if (s == range_start(c + 1, jobs.G, total)) continue;  // an empty range
      // the job is the CTA's first one unless the CTA began with an earlier job
      const int64_t slot = 2 * static_cast<int64_t>(c) + (s < start ? 1 : 0);
      const float2 w = ws.ml[slot * kH + h];
      if (w.x == -INFINITY && w.y == 0.f) continue;  // no row of it counts (a NaN sum does)
      const float4 v = reinterpret_cast<const float4 *>(ws.o + (slot * kH + h) * kD + 128 * quarter)[lane];
      const float mn = fmaxf(m, w.x), f = m == mn ? 1.f : exp2f(m - mn), e = w.x == mn ? 1.f : exp2f(w.x - mn);
      l = fmaf(l, f, e * w.y);
      acc.x = fmaf(acc.x, f, e * v.x);
      acc.y = fmaf(acc.y, f, e * v.y);
      acc.z = fmaf(acc.z, f, e * v.z);
      acc.w = fmaf(acc.w, f, e * v.w);
      m = mn;
    }
    __syncthreads();
    acc_s[warp][lane] = acc;
    if (lane == 0) ml_s[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) continue;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; w++) m = fmaxf(m, ml_s[w].x);
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMergeThreads / 32; w++) {
      const float2 x = ml_s[w];
      if (x.x == -INFINITY && x.y == 0.f) continue;
      const float e = x.x == m ? 1.f : exp2f(x.x - m);
      const float4 v = acc_s[w][lane];
      l = fmaf(e, x.y, l);
      acc.x = fmaf(e, v.x, acc.x);
      acc.y = fmaf(e, v.y, acc.y);
      acc.z = fmaf(e, v.z, acc.z);
      acc.w = fmaf(e, v.w, acc.w);
    }
    const float il = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = static_cast<int64_t>(bt) * a.H + group * kH + h;
    const uint2 o = make_uint2(bf16_bits(acc.x * il) | (bf16_bits(acc.y * il) << 16),
                               bf16_bits(acc.z * il) | (bf16_bits(acc.w * il) << 16));
    reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * kD + 128 * quarter)[lane] = o;
    if (a.lse && quarter == 0 && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
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
  j.groups = (a.H + kH - 1) / kH;
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
  return LIDX_WS_HEADER + align256(j.G * sizeof(Split)) + static_cast<size_t>(j.G) * 2 * kH * (8 + kD * 4);
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
  p += static_cast<size_t>(j.G) * 2 * kH * 8;
  s.o = reinterpret_cast<float *>(p);
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
