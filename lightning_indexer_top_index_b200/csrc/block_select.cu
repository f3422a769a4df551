// Block selection: the cheap score of every block a query sees, and the k
// blocks with the largest.
//
// Score.  A warp takes eight blocks at a time with mma.m16n8k32 (s8): the 64
// heads' 8-bit queries are the A operand, held in registers for the whole row
// (4 tiles of 16 heads x 4 steps of 32 dims); a block's 128 codes are the B
// operand, loaded as 32 bytes by each of four lanes (a dot product does not
// care which dims a step takes, so a lane's own 32 bytes are its share of all
// four steps).  The dots are whole numbers below 2^21.  Each lane folds its 8
// heads' ReLU'd dots with 64-bit weights and the 8 lanes of a block add up.  A
// dot becomes a double by its bits (2^52 + n, minus 2^52), which costs an add.
// A step is bound by the latency of its chain, so the four tiles' products are
// issued in turn, and the weights are read from shared memory, so that
// the products and the next step's codes have registers (32 rows of 128 blocks
// a CTA: 8.5 -> 8.0 us; with the codes of two steps ahead it gained nothing).
//
// Selection.  Scores become order-preserving 64-bit keys in shared memory
// (0: not eligible, all ones: always taken).  Few keys are ranked directly, a
// thread each.  More are binned linearly in value between the smallest and the
// largest score (the bin is a monotone function of the score, so the bin that
// holds the k-th largest and the count above it are exact), and the keys of
// that bin are ranked; where too many share it, a radix over 11-bit digits
// from the highest bit in which the keys differ finds the k-th largest.  Ids
// come out ascending by a prefix sum; equal keys are taken from the lowest
// index on.
//
// A row's blocks are split over a cluster of up to 16 CTAs when there are few
// rows; every CTA selects its k best, pushes them into the first CTA's shared
// memory, and that one selects among them in the same way (the slices are
// contiguous, so the lists stay in index order).
#include <algorithm>
#include <atomic>

#include "paged.cuh"
#include "tc.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxBlocks = 8 * 16384;  // of a sequence: what 8 CTAs hold, where the device has no clusters of 16
constexpr int kMaxSlice = 16384;  // keys a CTA holds
constexpr int kMaxK = 256;
constexpr int kDigit = 11, kBins = 1 << kDigit;
constexpr int kLinear = 512;      // bins of the scores' range (2048: 18.1 us for 512 rows of 256 blocks instead of 17.6)
constexpr int kLong = 8192;       // blocks of a row from which on more than four rows take clusters of 16
constexpr int kCand = 256;        // keys of a bin ranked directly
constexpr int kDirect = 128;      // keys of a row ranked directly without binning (with 64: 8.0 -> 8.5 us for 128
                                  // a CTA; with 256: 10.3 -> 12.4 us for 244)
constexpr int kPitch = 144;       // bytes between a head's codes: 16-byte reads of 8 heads x 4 lanes hit all banks
constexpr uint64_t kForced = ~0ull;

struct Smem {
  alignas(16) uint8_t q[64 * kPitch];
  double weight[64];
  uint32_t hist[kBins];
  uint64_t cand[kCand];
  uint64_t red_or[kWarps], red_and[kWarps];
  uint32_t scan_a[kWarps], scan_b[kWarps];
  uint32_t n_cand, bin, above, bin_count;
  float red_lo[kWarps], red_hi[kWarps];
  uint32_t red_some[kWarps], red_must[kWarps];
  int32_t picked[kMaxK];
  uint64_t threshold;
  uint32_t need;
  // the first CTA's side of the exchange
  uint32_t in_count[kMaxCluster];
};

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ double whole(int n) {  // n in [0, 2^31)
  return __hiloint2double(0x43300000, n) - 4503599627370496.0;
}

// larger double -> larger key in [1, kForced), -0 as +0; NaN -> 0.  No finite
// or infinite double reaches kForced (it would be a NaN).
__device__ __forceinline__ uint64_t key_of(double s) {
  if (s != s) return 0ull;
  if (s == 0.) s = 0.;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(s));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t remote(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(p)), "r"(rank));
  return a;
}

// exclusive prefix sums of (x, y) over the CTA's threads, and the totals
__device__ __forceinline__ void scan2(Smem &sm, uint32_t x, uint32_t y, uint32_t &px, uint32_t &py, uint32_t &tx,
                                      uint32_t &ty) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ix = warp_inclusive_scan(x), iy = warp_inclusive_scan(y);
  __syncthreads();
  if (lane == 31) {
    sm.scan_a[warp] = ix;
    sm.scan_b[warp] = iy;
  }
  __syncthreads();
  px = ix - x;
  py = iy - y;
  tx = ty = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    const uint32_t u = sm.scan_a[w], v = sm.scan_b[w];
    if (w < warp) {
      px += u;
      py += v;
    }
    tx += u;
    ty += v;
  }
}

__device__ __forceinline__ bool ranked(uint64_t key) { return key + 1ull > 1ull; }  // neither 0 nor kForced

__device__ __forceinline__ float value_of(uint64_t key) {  // monotone in the key
  const uint64_t u = (key >> 63) ? key & 0x7FFFFFFFFFFFFFFFull : ~key;
  return static_cast<float>(__longlong_as_double(static_cast<long long>(u)));
}

// The bin that holds the want-th largest of sm.hist's `bins` counted keys,
// from above: sm.bin, sm.above (keys in the bins above it), sm.bin_count.
template <int kN>
__device__ __forceinline__ void find_bin(Smem &sm, uint32_t want) {
  constexpr int per = kN / kThreads;
  const int tid = threadIdx.x;  // thread t sums bins from the top on
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < per; i++) mine += sm.hist[kN - 1 - (tid * per + i)];
  uint32_t before, zero, total, zero2;
  scan2(sm, mine, 0u, before, zero, total, zero2);
  if (before < want && want <= before + mine) {
    uint32_t at = before;
    for (int i = 0; i < per; i++) {
      const int bin = kN - 1 - (tid * per + i);
      const uint32_t h = sm.hist[bin];
      if (want <= at + h) {
        sm.bin = bin;
        sm.above = at;
        sm.bin_count = h;
        break;
      }
      at += h;
    }
  }
  __syncthreads();
}

// The want-th largest of the sm.n_cand <= kCand keys in sm.cand: sm.threshold,
// and in sm.need how many keys equal to it belong to the `want` largest.
__device__ __forceinline__ void rank_candidates(Smem &sm, uint32_t want) {
  const int tid = threadIdx.x, nc = sm.n_cand;
  if (tid < nc) {
    const uint64_t x = sm.cand[tid];
    uint32_t above = 0, same = 0;
    for (int i = 0; i < nc; i++) {
      above += sm.cand[i] > x;
      same += sm.cand[i] == x;
    }
    if (above < want && want <= above + same) {  // all threads with this value write the same
      sm.threshold = x;
      sm.need = want - above;
    }
  }
  __syncthreads();
}

// The k-th largest (k >= 1) of those of the n keys that are neither 0 nor
// kForced, of which there are `count` > k, by radix: sm.threshold and sm.need.
__device__ __noinline__ void kth_by_radix(Smem &sm, const uint64_t *keys, int n, uint32_t count, uint32_t k) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t any = 0ull, all = ~0ull;
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t x = keys[i];
    if (ranked(x)) {
      any |= x;
      all &= x;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    any |= __shfl_xor_sync(0xFFFFFFFFu, any, o);
    all &= __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  if (lane == 0) {
    sm.red_or[warp] = any;
    sm.red_and[warp] = all;
  }
  __syncthreads();
  any = 0ull;
  all = ~0ull;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    any |= sm.red_or[w];
    all &= sm.red_and[w];
  }
  const uint64_t differ = any ^ all;
  int top = differ ? 64 - __clzll(static_cast<long long>(differ)) : 0;  // bits [0, top) may differ
  uint64_t prefix = top < 64 ? (all >> top) : 0ull;                     // the k-th key's bits from `top` on
  uint32_t want = k;                                                    // its rank among the `count` keys with that prefix
  while (top > 0 && count > kCand) {
    const int shift = max(top - kDigit, 0), bins = 1 << (top - shift);
    for (int i = tid; i < kBins; i += kThreads) sm.hist[i] = 0u;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t x = keys[i];
      if (ranked(x) && (top == 64 || (x >> top) == prefix))
        atomicAdd(&sm.hist[static_cast<uint32_t>(x >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    find_bin<kBins>(sm, want);
    prefix = (top == 64 ? 0ull : prefix << (top - shift)) | sm.bin;
    want -= sm.above;
    count = sm.bin_count;
    top = shift;
    __syncthreads();
  }
  if (top == 0) {  // every remaining key is the same
    if (tid == 0) {
      sm.threshold = prefix;
      sm.need = want;
    }
    __syncthreads();
    return;
  }
  if (tid == 0) sm.n_cand = 0u;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t x = keys[i];
    if (ranked(x) && (top == 64 || (x >> top) == prefix)) sm.cand[atomicAdd(&sm.n_cand, 1u)] = x;
  }
  __syncthreads();
  rank_candidates(sm, want);
}

// The same, with the scores binned linearly between lo and hi first.
__device__ __forceinline__ void kth_largest(Smem &sm, const uint64_t *keys, int n, uint32_t count, uint32_t k, float lo,
                                            float hi) {
  const int tid = threadIdx.x;
  // infinities, NaN ranges and equal scores: everything in bin 0
  float per_bin = (kLinear - 1) / (hi - lo);
  if (!(per_bin < 3e38f) || !(hi - lo < 3e38f)) per_bin = 0.f;
  auto bin_of = [&](uint64_t key) {
    return min(max(static_cast<int>((value_of(key) - lo) * per_bin), 0), kLinear - 1);
  };
  for (int i = tid; i < kLinear; i += kThreads) sm.hist[i] = 0u;
  if (tid == 0) sm.n_cand = 0u;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads)
    if (ranked(keys[i])) atomicAdd(&sm.hist[bin_of(keys[i])], 1u);
  __syncthreads();
  find_bin<kLinear>(sm, k);
  if (sm.bin_count > kCand) {
    kth_by_radix(sm, keys, n, count, k);
    return;
  }
  const int bin = sm.bin;
  for (int i = tid; i < n; i += kThreads)
    if (ranked(keys[i]) && bin_of(keys[i]) == bin) sm.cand[atomicAdd(&sm.n_cand, 1u)] = keys[i];
  __syncthreads();
  rank_candidates(sm, k - sm.above);
}

// What the selection needs to know about a CTA's keys.
struct Keys {
  int n;
  uint32_t some, must;  // eligible ones, and of them those always taken
  float lo, hi;         // the range of the others' scores
};

// The indexes of the k largest of keys[0..n) (ties to the lower index), in
// ascending order into sm.picked; returns how many there are.  (Not inlined:
// the code is used in two places and fetching it is what a short call pays.)
__device__ __noinline__ int select_k(Smem &sm, const uint64_t *keys, const Keys in, int k) {
  const int tid = threadIdx.x, n = in.n;
  if (n <= kDirect) {
    bool taken = false;
    if (tid < n) {
      const uint64_t x = keys[tid];
      int rank = 0;
#pragma unroll 4
      for (int i = 0; i < n; i++) {
        const uint64_t y = keys[i];
        rank += y > x || (y == x && i < tid);
      }
      taken = x != 0ull && rank < k;
    }
    const uint32_t flags = __ballot_sync(0xFFFFFFFFu, taken);
    if ((tid & 31) == 0) sm.scan_a[tid >> 5] = __popc(flags);
    __syncthreads();
    int slot = __popc(flags & ((1u << (tid & 31)) - 1u)), total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      if (w < (tid >> 5)) slot += sm.scan_a[w];
      total += sm.scan_a[w];
    }
    if (taken) sm.picked[slot] = tid;
    __syncthreads();
    return total;
  }
  const bool all = in.some <= static_cast<uint32_t>(k);
  uint64_t T = 0ull;  // keys > T are taken, and `need` of those equal to it
  uint32_t need = 0;
  if (!all && in.must >= static_cast<uint32_t>(k)) {
    T = kForced;
    need = k;
  } else if (!all) {
    kth_largest(sm, keys, n, in.some - in.must, k - in.must, in.lo, in.hi);
    T = sm.threshold;
    need = sm.need;
  }
  const int per = (n + kThreads - 1) / kThreads, lo = min(tid * per, n), hi = min(lo + per, n);
  uint32_t gt = 0, eq = 0;
  for (int i = lo; i < hi; i++) {
    gt += keys[i] > T;
    eq += keys[i] == T;
  }
  uint32_t pg, pe, tg, te;
  scan2(sm, gt, eq, pg, pe, tg, te);
  uint32_t slot = pg + min(pe, need);
  for (int i = lo; i < hi; i++) {
    const uint64_t x = keys[i];
    if (x > T || (x == T && pe < need)) sm.picked[slot++] = i;
    pe += x == T;
  }
  __syncthreads();
  return static_cast<int>(all ? in.some : static_cast<uint32_t>(k));
}

// (two CTAs an SM: with six registers more a thread and one CTA, 512 rows took
// 29 us instead of 19)
__global__ void __launch_bounds__(kThreads, 2) block_select_kernel(const lidx_block_select_args a, int G, int shift,
                                                                 int slice_cap, uint32_t *status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
  uint64_t *keys = reinterpret_cast<uint64_t *>(smem_raw + sizeof(Smem));  // [slice_cap], then the exchange's lists
  const int rank = G > 1 ? static_cast<int>(cluster_rank()) : 0;
  uint64_t *in_key = keys + slice_cap;                               // [G * k]
  int32_t *in_id = reinterpret_cast<int32_t *>(in_key + G * a.k);    // [G * k]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bt = blockIdx.x / G;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt % a.T);
  if (G > 1) cluster_arrive();
  pdl_trigger();
  pdl_wait();

  // ---- this CTA's blocks [j0, j1) of the nb that the query sees; the first ones' codes are fetched
  // while the queries are rounded
  const int g = lane >> 2, c = lane & 3;
  const int64_t most = static_cast<int64_t>(a.max_pages) << shift;
  const int32_t len_in = fetch(a.len + b);
  const int qh = tid >> 2, qc = tid & 3;  // queries: thread (head, quarter) owns 32 dims
  uint4 qw[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    qw[i] = make_uint4(0, 0, 0, 0);
    if (qh < a.H)
      qw[i] = fetch(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + (bt * a.H + qh) * 128 + 32 * qc) + i);
  }
  const float qweight = qh < a.H ? fetch(a.w + bt * a.H + qh) : 0.f;
  if (len_in > most && rank == 0 && tid == 0) raise_status(status, LIDX_DEV_BOUNDS);
  const int64_t seen = min(static_cast<int64_t>(max(len_in, 0)), most) - (a.T - 1 - t);
  const int nb = seen > 0 ? static_cast<int>((seen + a.page_rows - 1) >> shift) : 0;
  const int per = ((nb + G - 1) / G + 7) & ~7;
  const int j0 = min(rank * per, nb), j1 = min(j0 + per, nb);
  const int32_t *table = a.table + static_cast<int64_t>(b) * a.ld_table;
  bool no_page = false, not_a_number = false;
  auto page_at = [&](int j) {  // of block j, -1 where there is none
    if (j >= j1) return -1;
    const int32_t p = fetch(table + j);
    return p;
  };
  struct Codes {
    uint4 x, y;  // bytes [32 c, 32 c + 32)
    float scale;
    int32_t page;
  };
  auto codes_of = [&](int32_t p, bool exists) {
    Codes k;
    k.x = k.y = make_uint4(0, 0, 0, 0);
    k.scale = 0.f;
    k.page = p < 0 || p >= a.n_pages ? -1 : p;
    no_page |= exists && k.page < 0;
    if (k.page >= 0) {
      const uint4 *src = reinterpret_cast<const uint4 *>(a.codes + static_cast<int64_t>(k.page) * 128 + 32 * c);
      k.x = fetch(src);
      k.y = fetch(src + 1);
      k.scale = fetch(a.scale + k.page);
    }
    return k;
  };
  // blocks j + g (lane (g, c)) of the steps j = j0 + 8 warp, + 8 kWarps, ..: two pages and one step's codes ahead
  const int first = j0 + 8 * warp + g;
  int32_t page1 = page_at(first);
  Codes now = codes_of(page1, first < j1);
  page1 = page_at(first + 8 * kWarps);

  // ---- the row's queries in 8 bits
  {
    const int h = qh, c = qc;
    float v[32], top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t x[4] = {qw[i].x, qw[i].y, qw[i].z, qw[i].w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        v[8 * i + 2 * k] = bf16x2_lo(x[k]);
        v[8 * i + 2 * k + 1] = bf16x2_hi(x[k]);
      }
    }
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      top = fmaxf(top, fabsf(v[i]));
      nan |= v[i] != v[i];
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (nan) top = __uint_as_float(0x7FC00000u);
    const bool bad = __shfl_xor_sync(0xFFFFFFFFu, nan, 1) | nan;
    if (__shfl_xor_sync(0xFFFFFFFFu, bad, 2) | bad) top = __uint_as_float(0x7FC00000u);
    float unit = top;
    if (top < 0x1p-100f) {  // 127 / top would leave the range of fp32
      unit *= 0x1p100f;
#pragma unroll
      for (int i = 0; i < 32; i++) v[i] *= 0x1p100f;
    }
    const float inv = unit > 0.f ? __fmul_rn(__frcp_rn(unit), 127.f) : 0.f;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      uint32_t r = 0;
#pragma unroll
      for (int k = 0; k < 4; k++)
        r |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(v[4 * i + k], inv))) & 0xFFu) << (8 * k);
      w[i] = r;
    }
    uint4 *dst = reinterpret_cast<uint4 *>(sm.q + h * kPitch + 32 * c);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (c == 0)
      sm.weight[h] = h < a.H ? static_cast<double>(__fmul_rn(qweight, __fmul_rn(top, 1.f / 127.f))) : 0.;
  }
  __syncthreads();
  uint32_t A[4][4][4];  // [tile][step][register]
#pragma unroll
  for (int m = 0; m < 4; m++) {
#pragma unroll
    for (int half = 0; half < 2; half++) {
      const int h = 16 * m + 8 * half + g;
      const uint4 *src = reinterpret_cast<const uint4 *>(sm.q + h * kPitch + 32 * c);
      const uint4 x = src[0], y = src[1];
      A[m][0][half] = x.x; A[m][0][2 + half] = x.y;
      A[m][1][half] = x.z; A[m][1][2 + half] = x.w;
      A[m][2][half] = y.x; A[m][2][2 + half] = y.y;
      A[m][3][half] = y.z; A[m][3][2 + half] = y.w;
    }
  }

  // ---- scores
  const int heads_tiles = (a.H + 15) / 16;
  const volatile double *weight = sm.weight + g;
  float lo = INFINITY, hi = -INFINITY;
  uint32_t some = 0, must = 0;
#pragma unroll 1
  for (int j = j0 + 8 * warp; j < j1; j += 8 * kWarps) {
    const Codes k = now;
    now = codes_of(page1, j + 8 * kWarps + g < j1);
    page1 = page_at(j + 16 * kWarps + g);
    const uint4 x = k.x, y = k.y;
    // lane (g, c) ends with heads g, g + 8 of each tile for blocks j + 2c, j + 2c + 1
    double s0 = 0., s1 = 0.;
    int d[4][4] = {};
    // the tiles' products in turn, as each step of a tile waits for the one before
    if (heads_tiles > 2) {
#pragma unroll
      for (int m = 0; m < 4; m++) mma_s8(d[m], A[m][0], x.x, x.y);
#pragma unroll
      for (int m = 0; m < 4; m++) mma_s8(d[m], A[m][1], x.z, x.w);
#pragma unroll
      for (int m = 0; m < 4; m++) mma_s8(d[m], A[m][2], y.x, y.y);
#pragma unroll
      for (int m = 0; m < 4; m++) mma_s8(d[m], A[m][3], y.z, y.w);
    } else {
#pragma unroll
      for (int m = 0; m < 2; m++) mma_s8(d[m], A[m][0], x.x, x.y);
#pragma unroll
      for (int m = 0; m < 2; m++) mma_s8(d[m], A[m][1], x.z, x.w);
#pragma unroll
      for (int m = 0; m < 2; m++) mma_s8(d[m], A[m][2], y.x, y.y);
#pragma unroll
      for (int m = 0; m < 2; m++) mma_s8(d[m], A[m][3], y.z, y.w);
    }
    double r0 = 0., r1 = 0.;
#pragma unroll
    for (int m = 0; m < 4; m++) {
      const double wa = weight[16 * m], wb = weight[16 * m + 8];
      s0 = fma(whole(max(d[m][0], 0)), wa, s0);
      s1 = fma(whole(max(d[m][1], 0)), wa, s1);
      r0 = fma(whole(max(d[m][2], 0)), wb, r0);
      r1 = fma(whole(max(d[m][3], 0)), wb, r1);
    }
    s0 += r0;
    s1 += r1;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
    }
    // lane (g, 0..3) < 8: block j + lane; its sum sits in s0 / s1 of lane c = lane / 2, its scale and page in lane 4 * lane
    const double sa = __shfl_sync(0xFFFFFFFFu, s0, (lane & 7) >> 1), sb = __shfl_sync(0xFFFFFFFFu, s1, (lane & 7) >> 1);
    const float sc = __shfl_sync(0xFFFFFFFFu, k.scale, 4 * (lane & 7));
    const int32_t pg = __shfl_sync(0xFFFFFFFFu, k.page, 4 * (lane & 7));
    const int jl = j + lane;
    if (lane < 8 && jl < j1) {
      const double score = ((lane & 1) ? sb : sa) * static_cast<double>(sc);
      uint64_t key = pg >= 0 ? key_of(score) : 0ull;
      if (jl < a.n_first || jl >= nb - a.n_last) {
        key = kForced;
        must++;
      } else if (key) {
        lo = fminf(lo, static_cast<float>(score));
        hi = fmaxf(hi, static_cast<float>(score));
      } else if (pg >= 0) {
        not_a_number = true;
      }
      some += key != 0ull;
      keys[jl - j0] = key;
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {  // lanes 0-7
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    some += __shfl_xor_sync(0xFFFFFFFFu, some, o);
    must += __shfl_xor_sync(0xFFFFFFFFu, must, o);
  }
  if (lane == 0) {
    sm.red_lo[warp] = lo;
    sm.red_hi[warp] = hi;
    sm.red_some[warp] = some;
    sm.red_must[warp] = must;
  }
  if (no_page) raise_status(status, LIDX_DEV_BOUNDS);
  if (not_a_number) raise_status(status, LIDX_DEV_NAN);
  __syncthreads();
  Keys mine_in = {j1 - j0, 0u, 0u, INFINITY, -INFINITY};
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    mine_in.some += sm.red_some[w];
    mine_in.must += sm.red_must[w];
    mine_in.lo = fminf(mine_in.lo, sm.red_lo[w]);
    mine_in.hi = fmaxf(mine_in.hi, sm.red_hi[w]);
  }

  int32_t *ids = a.ids + bt * a.k;
  int n_sel = select_k(sm, keys, mine_in, a.k);
  int32_t id = tid < n_sel ? j0 + sm.picked[tid] : -1;  // kMaxK <= kThreads
  if (G > 1) {
    cluster_wait();  // the first CTA runs: its shared memory may be written
    const int mine = n_sel;
    if (tid < mine) {
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(in_key + rank * a.k + tid, 0)), "l"(keys[id - j0])
                   : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(in_id + rank * a.k + tid, 0)), "r"(id) : "memory");
    }
    if (tid == 0)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(&sm.in_count[rank], 0)), "r"(mine) : "memory");
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    // the lists close up in place, in index order (list r moves down to the end of list r - 1)
    int n = sm.in_count[0];
    for (int r = 1; r < G; r++) {
      const int cnt = sm.in_count[r];
      uint64_t key = 0;
      int32_t one = 0;
      if (tid < cnt) {
        key = in_key[r * a.k + tid];
        one = in_id[r * a.k + tid];
      }
      __syncthreads();
      if (tid < cnt) {
        in_key[n + tid] = key;
        in_id[n + tid] = one;
      }
      n += cnt;
    }
    // (every entry is eligible; the range of their scores, from the lists)
    Keys all_in = {n, static_cast<uint32_t>(n), 0u, INFINITY, -INFINITY};
    __syncthreads();
    if (n > kDirect) {
      lo = INFINITY;
      hi = -INFINITY;
      must = 0;
      for (int i = tid; i < n; i += kThreads) {
        if (ranked(in_key[i])) {
          lo = fminf(lo, value_of(in_key[i]));
          hi = fmaxf(hi, value_of(in_key[i]));
        } else {
          must++;
        }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        must += __shfl_xor_sync(0xFFFFFFFFu, must, o);
      }
      if (lane == 0) {
        sm.red_lo[warp] = lo;
        sm.red_hi[warp] = hi;
        sm.red_must[warp] = must;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        all_in.must += sm.red_must[w];
        all_in.lo = fminf(all_in.lo, sm.red_lo[w]);
        all_in.hi = fmaxf(all_in.hi, sm.red_hi[w]);
      }
    }
    n_sel = select_k(sm, in_key, all_in, a.k);
    id = tid < n_sel ? in_id[sm.picked[tid]] : -1;
  }
  if (tid < a.k) ids[tid] = id;
  if (tid == 0 && a.n_sel) a.n_sel[bt] = n_sel;
}

constexpr size_t smem_of(int g, int slice, int k) {
  return sizeof(Smem) + static_cast<size_t>(slice) * 8 + (g > 1 ? static_cast<size_t>(g) * k * 12 : 0);
}

static_assert(smem_of(16, kMaxBlocks / 16, kMaxK) <= smem_of(8, kMaxSlice, kMaxK), "the largest is a cluster of 8's");

// The same for every call of the process, so that calls from several threads agree.
cudaError_t allow_largest() {
  const cudaError_t e = allow_smem(block_select_kernel, smem_of(8, kMaxSlice, kMaxK));  // a cluster of 16 needs less
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(block_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// Does the current device run clusters of 16 CTAs, as large as they get here?
bool cluster16_ok() {
  static std::atomic<int> cache[64];  // by device: 0 not asked yet, 1 yes, 2 no
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return false;
  }
  int known = cache[dev].load(std::memory_order_relaxed);
  if (!known) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_of(16, kMaxBlocks / 16, kMaxK);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = allow_largest() == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, block_select_kernel, &cfg) == cudaSuccess && n >= 1;
    cudaGetLastError();
    known = ok ? 1 : 2;
    cache[dev].store(known, std::memory_order_relaxed);
  }
  return known == 1;
}

// CTAs a row is split over: so that a slice fits, and, while the rows leave
// SMs idle, down to 128 blocks a CTA.  Sixteen for one to four rows (1954
// blocks: 10.5 -> 9.9 us, 62500: 87 -> 53), and for up to nine long ones (9 x
// 14000: 26.2 -> 23.6; 9 x 2000 would go from 10.7 to 11.9).
int cluster_for(const lidx_block_select_args &a) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.T;
  int g = 1;
  while (g < 8 && (a.max_pages > g * kMaxSlice || (a.max_pages > g * 128 && rows * g * 2 <= 148))) g *= 2;
  if (g == 8 && a.max_pages > 8 * 128 && rows * 16 <= 148 && (rows <= 4 || a.max_pages > kLong) && cluster16_ok()) g = 16;
  return g;
}

int slice_of(const lidx_block_select_args &a, int g) { return ((a.max_pages + g - 1) / g + 7) & ~7; }

}  // namespace

bool block_select_supported(const lidx_block_select_args &a) {
  return a.k <= kMaxK && a.H <= 64 && a.max_pages <= kMaxBlocks;
}

cudaError_t launch_block_select(const lidx_block_select_args &a, void *ws, cudaStream_t st) {
  const int g = cluster_for(a), slice = slice_of(a, g);
  const size_t smem = smem_of(g, slice, a.k);
  const cudaError_t e = allow_largest();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(g * a.B * a.T));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (g > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = g;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    n++;
  }
  if (a.flags & LIDX_LAUNCH_PDL) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    n++;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, block_select_kernel, a, g, __builtin_ctz(static_cast<unsigned>(a.page_rows)), slice,
                            static_cast<uint32_t *>(ws));
}

}  // namespace lidx
