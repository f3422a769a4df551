// The paged cache's write side, and rows read back.
//
// Append: a new row's last 64 dims are rotated in pairs by the angles
// pos * inv_freq[i], the others rounded to E4M3 or E2M1 under one power-of-two
// scale per 64 or 32 of them, and the row goes to its page.
//
// A row is served by a warp, or by eight lanes for an index key.  A lane has a
// share of the dims that are rounded (16 of 28 lanes, or 8 of eight) and, of the
// rotated ones, the pairs whose angles it evaluates (one, or four), so that no
// value or angle is handed from lane to lane: with the rotated dims held 16 a
// lane by four lanes and their angles fetched by shuffles, 20011 rows of 512,
// appended and read back, took 28.4 us instead of 25.6.  An angle is formed as
// pos * inv_freq / 2 pi turns in 64 bits and its whole turns dropped before it
// is rounded to fp32 (error below 2^-25 turns up to 2^25 of them, from there on
// 2^-51 of the turns), since in fp32 the product alone would be off by up to
// pos * 2^-24 radians.
#include "paged.cuh"
#include "quant.cuh"

namespace lidx {

namespace {

constexpr int kThreads = 128;
constexpr unsigned kAll = 0xFFFFFFFFu;

// N adjacent values, at a multiple of N of a row (of 4, 2 or 1 for smaller ones).
template <int N>
__device__ __forceinline__ void load_values(const void *x, int dtype, int64_t at, float *v) {
  if (dtype == LIDX_F32) {
    const float *s = static_cast<const float *>(x) + at;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; i++) {
        const float4 a = fetch(reinterpret_cast<const float4 *>(s) + i);
        v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
      }
    } else if constexpr (N == 2) {
      const float2 a = fetch(reinterpret_cast<const float2 *>(s));
      v[0] = a.x; v[1] = a.y;
    } else {
      v[0] = fetch(s);
    }
  } else {
    const uint16_t *s = static_cast<const uint16_t *>(x) + at;
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N / 8; i++) {
        const uint4 a = fetch(reinterpret_cast<const uint4 *>(s) + i);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
          v[8 * i + 2 * k] = bf16x2_lo(w[k]);
          v[8 * i + 2 * k + 1] = bf16x2_hi(w[k]);
        }
      }
    } else if constexpr (N == 4) {
      const uint2 a = fetch(reinterpret_cast<const uint2 *>(s));
      v[0] = bf16x2_lo(a.x); v[1] = bf16x2_hi(a.x); v[2] = bf16x2_lo(a.y); v[3] = bf16x2_hi(a.y);
    } else if constexpr (N == 2) {
      const uint32_t a = fetch(reinterpret_cast<const uint32_t *>(s));
      v[0] = bf16x2_lo(a); v[1] = bf16x2_hi(a);
    } else {
      v[0] = bf16x2_lo(fetch(s));
    }
  }
}

template <int N>
__device__ __forceinline__ void store_f32(float *o, const float *v) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; i++)
      reinterpret_cast<float4 *>(o)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2 *>(o) = make_float2(v[0], v[1]);
  } else {
    o[0] = v[0];
  }
}

// `odd`: some may be NaN
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *o, const float *v, bool odd) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; i++)
      reinterpret_cast<uint4 *>(o)[i] = odd ? pack8_bf16(v + 8 * i) : pack8_bf16_numbers(v + 8 * i);
  } else if constexpr (N == 1) {
    o[0] = static_cast<uint16_t>(bf16_bits(v[0]));
  } else {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; i++) w[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
    if constexpr (N == 4) *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(o) = w[0];
  }
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

template <int kDim>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const lidx_paged_append_args a, int shift,
                                                                 uint32_t *status) {
  constexpr int kLanes = kDim / 16;            // lanes of a row
  constexpr int kPairs = 32 / kLanes;          // pairs, and angles, of a lane
  constexpr int kN = kDim == 512 ? 16 : 8;     // a lane's other dims
  constexpr int kHolders = (kDim - 64) / kN;   // lanes that have some
  const int t = threadIdx.x % kLanes;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  const bool holds = t < kHolders, adjacent = a.rope_pairs == LIDX_ROPE_ADJACENT;
  // the lane's pairs: their first values from dim u0, and, by halves, their second ones from dim u0 + 32
  const int u0 = kDim - 64 + (adjacent ? 2 : 1) * kPairs * t;
  pdl_trigger();
  pdl_wait();  // rows, positions and tables may come from the previous kernel
  // lanes of rows behind the last one stay for the shuffles
  int seq = -1, row = -1, pos = 0;
  float x[kN], r[2 * kPairs], freq[kPairs];  // r: as stored, (u, v) pairs or the u's and then the v's
#pragma unroll
  for (int k = 0; k < kN; k++) x[k] = 0.f;
#pragma unroll
  for (int k = 0; k < 2 * kPairs; k++) r[k] = 0.f;
  if (i < a.n) {
    seq = fetch(a.seq + i);
    row = fetch(a.row + i);
    if (a.inv_freq) pos = a.pos ? fetch(a.pos + i) : row;
    if (holds) load_values<kN>(a.x, a.x_dtype, i * a.ld_x + kN * t, x);
    if (adjacent) {
      load_values<2 * kPairs>(a.x, a.x_dtype, i * a.ld_x + u0, r);
    } else {
      load_values<kPairs>(a.x, a.x_dtype, i * a.ld_x + u0, r);
      load_values<kPairs>(a.x, a.x_dtype, i * a.ld_x + u0 + 32, r + kPairs);
    }
  }
  if (a.inv_freq) {
#pragma unroll
    for (int k = 0; k < kPairs; k++) freq[k] = fetch(a.inv_freq + t * kPairs + k);
  }
  int32_t dst = -1;
  if (seq >= 0) {
    if (seq < a.B && row >= 0) dst = pool_row(a.cache, shift, seq, row);
    if (dst < 0 && t == 0) raise_status(status, LIDX_DEV_BOUNDS);
  }
  // the largest magnitude by its bits; infinities and NaNs have the largest
  uint32_t top = 0u, top_r = 0u;
#pragma unroll
  for (int k = 0; k < kN; k++) top = max(top, magnitude(x[k]));
#pragma unroll
  for (int k = 0; k < 2 * kPairs; k++) top_r = max(top_r, magnitude(r[k]));
  const bool nonfinite = max(top, top_r) >= 0x7F800000u;
  if (nonfinite && dst >= 0) raise_status(status, LIDX_DEV_NAN);
  const bool odd = __any_sync(kAll, nonfinite);  // the warp's rows take the careful way
  if (odd) {
    top = 0u;
#pragma unroll
    for (int k = 0; k < kN; k++) top = isfinite(x[k]) ? max(top, magnitude(x[k])) : top;
  }
  // ... of the block: the lanes that hold its 64 or 32 dims
  const int dtype = a.cache.rows.dtype;
  constexpr int kShare = 32 / kN;  // lanes of 32 dims
#pragma unroll
  for (int o = 1; o < kShare; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
  if (dtype == LIDX_E4M3) top = max(top, __shfl_xor_sync(kAll, top, kShare));

  if (a.inv_freq) {
#pragma unroll
    for (int k = 0; k < kPairs; k++) {
      double turns = static_cast<double>(pos) * static_cast<double>(freq[k]) * 0.15915494309189533577;
      turns -= rint(turns);
      float s, c;
      sincospif(2.f * static_cast<float>(turns), &s, &c);
      float &u = r[adjacent ? 2 * k : k], &v = r[adjacent ? 2 * k + 1 : kPairs + k];
      const float p = u, q = v;
      u = fmaf(p, c, -(q * s));
      v = fmaf(p, s, q * c);
    }
  }

  if (dst < 0) return;

  const lidx_kv &kv = a.cache.rows;
  const int64_t p = dst;
  // the rotated dims
  if (dtype == LIDX_F32) {
    float *o = static_cast<float *>(const_cast<void *>(kv.data)) + p * kv.ld;
    if (adjacent) {
      store_f32<2 * kPairs>(o + u0, r);
    } else {
      store_f32<kPairs>(o + u0, r);
      store_f32<kPairs>(o + u0 + 32, r + kPairs);
    }
    if (holds) store_f32<kN>(o + kN * t, x);
    return;
  }
  uint16_t *o = dtype == LIDX_BF16 ? static_cast<uint16_t *>(const_cast<void *>(kv.data)) + p * kv.ld
                                   : static_cast<uint16_t *>(const_cast<void *>(kv.rope)) + p * kv.ld_rope - (kDim - 64);
  if (adjacent) {
    store_bf16<2 * kPairs>(o + u0, r, odd);
  } else {
    store_bf16<kPairs>(o + u0, r, odd);
    store_bf16<kPairs>(o + u0 + 32, r + kPairs, odd);
  }
  if (!holds) return;
  if (dtype == LIDX_BF16) {
    store_bf16<kN>(o + kN * t, x, odd);
    return;
  }
  const bool e4m3 = dtype == LIDX_E4M3;
  const float am = __uint_as_float(top);
  const int e = top ? (e4m3 ? block_exponent_e4m3(am) : block_exponent_e2m1(am)) : 0;
  const float inv = inverse_scale(e);
#pragma unroll
  for (int k = 0; k < kN; k++) x[k] *= inv;
  uint8_t *data = static_cast<uint8_t *>(const_cast<void *>(kv.data)) + p * kv.ld;
  uint8_t *scale = const_cast<uint8_t *>(kv.scale) + p * kv.ld_scale;
  uint32_t w[kN / 4];
  if (e4m3) {
#pragma unroll
    for (int k = 0; k < kN / 4; k++) w[k] = odd ? pack4_e4m3(x + 4 * k) : pack4_e4m3_in_range(x + 4 * k);
    if constexpr (kN == 16) *reinterpret_cast<uint4 *>(data + 16 * t) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(data + 8 * t) = make_uint2(w[0], w[1]);
    if (t % (2 * kShare) == 0) scale[t / (2 * kShare)] = static_cast<uint8_t>(e + 127);
  } else {
#pragma unroll
    for (int k = 0; k < kN / 8; k++) w[k] = odd ? pack8_e2m1(x + 8 * k) : pack8_e2m1_finite(x + 8 * k);
    if constexpr (kN == 16) *reinterpret_cast<uint2 *>(data + 8 * t) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(data + 4 * t) = w[0];
    if (t % kShare == 0) scale[t / kShare] = static_cast<uint8_t>(e + 127);
  }
}

// Rows as values: dim/8 threads a row, thread t dims [8t, 8t + 8), kPer rows of
// it in flight together.  Instructions and loads bound it (65 % of the issue
// slots): as bf16 the values come from bf16 products of code and scale (through
// fp32, and rounded with a look for NaNs, the 20011 rows took 3 us more).
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
    if (kFmt != LIDX_F32 && a.out_dtype == LIDX_BF16) {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (i0 + r) * a.ld_out + 8 * t) =
          p[r] >= 0 ? raw[r].bf16() : make_uint4(0, 0, 0, 0);
      continue;
    }
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
// four (20011 rows of 512 in 4 bits, with their append: 22.5 us against 26.7
// with one; 64 rows 4.6 us with one and 5.3 with four).
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
