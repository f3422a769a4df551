// The paged cache's write side, and rows read back.
//
// Append: a new row's last 64 dims are rotated in pairs by the angles
// pos * inv_freq[i], the others rounded to E4M3 or E2M1 under one power-of-two
// scale per 64 or 32 of them, and the row goes to its page.
//
// A row is served by dim/16 lanes, lane t holding dims [16t, 16t + 16): a
// whole warp for a 512-wide row, eight lanes for an index key.  The row's 32
// angles are spread over its lanes (one, or four, each) and fetched by
// shuffles by the four lanes that hold the rotated dims, so no lane evaluates
// more than its share of sines.  An angle is formed as pos * inv_freq / 2 pi
// turns in 64 bits and its whole turns dropped before it is rounded to fp32
// (error below 2^-25 turns at any position), since in fp32 the product alone
// would be off by up to pos * 2^-24 radians.
#include "paged.cuh"
#include "quant.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ void load16(const void *x, int dtype, int64_t at, float (&v)[16]) {
  if (dtype == LIDX_F32) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(x) + at);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float4 a = fetch(s + i);
      v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
    }
  } else {
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint4 a = fetch(s + i);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; k++) {
        v[8 * i + 2 * k] = bf16x2_lo(w[k]);
        v[8 * i + 2 * k + 1] = bf16x2_hi(w[k]);
      }
    }
  }
}

template <int kDim>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const lidx_paged_append_args a, int shift,
                                                                 uint32_t *status) {
  constexpr int kLanes = kDim / 16;          // lanes of a row
  constexpr int kAngles = 32 / kLanes;       // angles a lane evaluates
  const int t = threadIdx.x % kLanes, lane = threadIdx.x & 31;
  const int base = lane - t;                 // the row's first lane
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const int rl = t - (kLanes - 4);  // >= 0: lane rl of the four that hold the 64 RoPE dims
  float freq[kAngles];
  pdl_trigger();
  pdl_wait();  // rows, positions and tables may come from the previous kernel
  // lanes of rows behind the last one stay for the shuffles
  int seq = -1, row = -1, pos = 0;
  float x[16];
#pragma unroll
  for (int k = 0; k < 16; k++) x[k] = 0.f;
  if (i < a.n) {
    seq = fetch(a.seq + i);
    row = fetch(a.row + i);
    if (a.inv_freq) pos = a.pos ? fetch(a.pos + i) : row;
    load16(a.x, a.x_dtype, i * a.ld_x + 16 * t, x);
  }
  if (a.inv_freq) {
#pragma unroll
    for (int k = 0; k < kAngles; k++) freq[k] = fetch(a.inv_freq + t * kAngles + k);
  }
  int32_t dst = -1;
  if (seq >= 0) {
    if (seq < a.B && row >= 0) dst = pool_row(a.cache, shift, seq, row);
    if (dst < 0 && t == 0) raise_status(status, LIDX_DEV_BOUNDS);
  }
  // the largest magnitude by its bits; infinities and NaNs have the largest
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < 16; k++) top = max(top, __float_as_uint(x[k]) & 0x7FFFFFFFu);
  const bool nonfinite = top >= 0x7F800000u;
  if (nonfinite && dst >= 0) raise_status(status, LIDX_DEV_NAN);
  const bool odd = __any_sync(kAll, nonfinite);  // the warp's rows take the careful way
  if (odd) {
    top = 0u;
#pragma unroll
    for (int k = 0; k < 16; k++) top = isfinite(x[k]) ? max(top, __float_as_uint(x[k]) & 0x7FFFFFFFu) : top;
  }
  // ... of the block: two or four neighbouring lanes
  const int dtype = a.cache.rows.dtype;
  top = max(top, __shfl_xor_sync(kAll, top, 1));
  if (dtype == LIDX_E4M3) top = max(top, __shfl_xor_sync(kAll, top, 2));

  if (a.inv_freq) {
    float cs[kAngles], sn[kAngles];
#pragma unroll
    for (int k = 0; k < kAngles; k++) {
      double turns = static_cast<double>(pos) * static_cast<double>(freq[k]) * 0.15915494309189533577;
      turns -= rint(turns);
      sincospif(2.f * static_cast<float>(turns), &sn[k], &cs[k]);
    }
    const int from = rl < 0 ? 0 : rl;
    if (a.rope_pairs == LIDX_ROPE_ADJACENT) {  // lane rl holds pairs 8 rl .. 8 rl + 7
#pragma unroll
      for (int k = 0; k < 8; k++) {
        // pair 8 rl + k: angle slot (8 rl + k) % kAngles of lane (8 rl + k) / kAngles
        const int src = base + (8 * from + k) / kAngles;
        const float c = __shfl_sync(kAll, cs[k % kAngles], src), s = __shfl_sync(kAll, sn[k % kAngles], src);
        if (rl >= 0) {
          const float p = x[2 * k], q = x[2 * k + 1];
          x[2 * k] = fmaf(p, c, -(q * s));
          x[2 * k + 1] = fmaf(p, s, q * c);
        }
      }
    } else {  // lanes 0, 1 hold the first halves of the pairs 16 (rl & 1) .. + 15, lanes 2, 3 their second halves
#pragma unroll
      for (int k = 0; k < 16; k++) {
        const int src = base + (16 * (from & 1) + k) / kAngles;
        const float c = __shfl_sync(kAll, cs[k % kAngles], src);
        const float s = __shfl_sync(kAll, sn[k % kAngles], src);
        const float o = __shfl_xor_sync(kAll, x[k], 2);
        if (rl >= 0) x[k] = rl < 2 ? fmaf(x[k], c, -(o * s)) : fmaf(o, s, x[k] * c);
      }
    }
  }

  if (dst < 0) return;

  const lidx_kv &kv = a.cache.rows;
  const int64_t p = dst;
  if (dtype == LIDX_F32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(const_cast<void *>(kv.data)) + p * kv.ld + 16 * t);
#pragma unroll
    for (int k = 0; k < 4; k++) o[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
  } else if (dtype == LIDX_BF16 || rl >= 0) {
    uint16_t *o = dtype == LIDX_BF16 ? static_cast<uint16_t *>(const_cast<void *>(kv.data)) + p * kv.ld + 16 * t
                                     : static_cast<uint16_t *>(const_cast<void *>(kv.rope)) + p * kv.ld_rope + 16 * rl;
    reinterpret_cast<uint4 *>(o)[0] = odd ? pack8_bf16(x) : pack8_bf16_numbers(x);
    reinterpret_cast<uint4 *>(o)[1] = odd ? pack8_bf16(x + 8) : pack8_bf16_numbers(x + 8);
  } else {
    const bool e4m3 = dtype == LIDX_E4M3;
    const float am = __uint_as_float(top);
    const int e = top ? (e4m3 ? block_exponent_e4m3(am) : block_exponent_e2m1(am)) : 0;
    const float inv = inverse_scale(e);
#pragma unroll
    for (int k = 0; k < 16; k++) x[k] *= inv;
    uint8_t *data = static_cast<uint8_t *>(const_cast<void *>(kv.data)) + p * kv.ld;
    uint8_t *scale = const_cast<uint8_t *>(kv.scale) + p * kv.ld_scale;
    if (e4m3) {
      *reinterpret_cast<uint4 *>(data + 16 * t) =
          odd ? make_uint4(pack4_e4m3(x), pack4_e4m3(x + 4), pack4_e4m3(x + 8), pack4_e4m3(x + 12))
              : make_uint4(pack4_e4m3_in_range(x), pack4_e4m3_in_range(x + 4), pack4_e4m3_in_range(x + 8),
                           pack4_e4m3_in_range(x + 12));
      if ((t & 3) == 0) scale[t / 4] = static_cast<uint8_t>(e + 127);
    } else {
      *reinterpret_cast<uint2 *>(data + 8 * t) = 
          odd ? make_uint2(pack8_e2m1(x), pack8_e2m1(x + 8))
              : make_uint2(pack8_e2m1_finite(x), pack8_e2m1_finite(x + 8));
      if ((t & 1) == 0) scale[t / 2] = static_cast<uint8_t>(e + 127);
    }
  }
}

// Rows as values: dim/8 threads a row, thread t dims [8t, 8t + 8), kPer rows of
// it in flight together.
template <int kFmt, int kPer>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const lidx_paged_read_args a, int shift,
                                                               uint32_t *status) {
  const int tpr = a.cache.rows.dim / 8, t = threadIdx.x % tpr;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / tpr) + threadIdx.x / tpr) * kPer;
  pdl_trigger();
  pdl_wait();
  int seq[kPer], row[kPer];
  int32_t p[kPer];
  Dims8<kFmt> raw[kPer];
#pragma unroll
  for (int r = 0; r < kPer; r++) {
    seq[r] = i0 + r < a.n ? fetch(a.seq + i0 + r) : -1;
    row[r] = i0 + r < a.n ? fetch(a.row + i0 + r) : -1;
  }
#pragma unroll
  for (int r = 0; r < kPer; r++)
    p[r] = seq[r] >= 0 && seq[r] < a.B && row[r] >= 0 ? pool_row(a.cache, shift, seq[r], row[r]) : -1;
#pragma unroll
  for (int r = 0; r < kPer; r++) {
    if (p[r] >= 0) raw[r].load(a.cache.rows, p[r], t);
    else if (seq[r] >= 0 && t == 0) raise_status(status, LIDX_DEV_BOUNDS);
  }
#pragma unroll
  for (int r = 0; r < kPer; r++) {
    if (seq[r] < 0) continue;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (p[r] >= 0) raw[r].values(v);
    if (a.out_dtype == LIDX_F32) {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + (i0 + r) * a.ld_out + 8 * t);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (i0 + r) * a.ld_out + 8 * t) = pack8_bf16(v);
    }
  }
}

// Blocks for n rows, `per` a group of `lanes` threads.
unsigned blocks(int64_t n, int lanes, int per) {
  const int64_t rows = static_cast<int64_t>(kThreads / lanes) * per;
  return static_cast<unsigned>((n + rows - 1) / rows);
}

}  // namespace

int page_shift(const lidx_pages &c) { return __builtin_ctz(static_cast<unsigned>(c.page_rows)); }

cudaError_t launch_paged_append(const lidx_paged_append_args &a, void *ws, cudaStream_t st) {
  auto kern = a.cache.rows.dim == 512 ? paged_append_kernel<512> : paged_append_kernel<128>;
  return launch_kernel(kern, dim3(blocks(a.n, a.cache.rows.dim / 16, 1)), dim3(kThreads), 0, st,
                       (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.cache), static_cast<uint32_t *>(ws));
}

// Few rows are read one a thread; from about a machine full of threads on,
// four (20011 rows of 512 in 4 bits: 13.1 us against 17.0 with one; 64 rows
// 4.0 us with one).
constexpr int64_t kManyThreads = 148 * 2048;

cudaError_t launch_paged_read(const lidx_paged_read_args &a, void *ws, cudaStream_t st) {
  const int lanes = a.cache.rows.dim / 8;
  const bool many = static_cast<int64_t>(a.n) * lanes >= kManyThreads;
  const int fmt = a.cache.rows.dtype;
  auto kern = many ? paged_read_kernel<LIDX_E2M1, 4> : paged_read_kernel<LIDX_E2M1, 1>;
  if (fmt == LIDX_E4M3) kern = many ? paged_read_kernel<LIDX_E4M3, 4> : paged_read_kernel<LIDX_E4M3, 1>;
  if (fmt == LIDX_BF16) kern = many ? paged_read_kernel<LIDX_BF16, 4> : paged_read_kernel<LIDX_BF16, 1>;
  if (fmt == LIDX_F32) kern = many ? paged_read_kernel<LIDX_F32, 4> : paged_read_kernel<LIDX_F32, 1>;
  return launch_kernel(kern, dim3(blocks(a.n, lanes, many ? 4 : 1)), dim3(kThreads), 0, st,
                       (a.flags & LIDX_LAUNCH_PDL) != 0, a, page_shift(a.cache), static_cast<uint32_t *>(ws));
}

}  // namespace lidx
